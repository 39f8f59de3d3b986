// Router: scores, group limit and top-k choice of every token in one launch.
//
// Source: P1 "Kimi 2.7 MoE: from 4-bit storage to INT8 (W4A8)" (pwwt.cn), section 4.1: the router stays in 16 bits,
// outside the quantized path, and hands the top-k ids and weights to the expert dispatch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "w4a8_device.h"
#include "w4a8_internal.h"

namespace w4a8 {

struct RouteArgs {
    const void* logits;
    int dtype;
    int T;
    long long ldl;
    const float* bias;
    int E, k, sigmoid, renorm, groups, keep;
    float scale;
    int32_t* ids;
    float* w;
};

constexpr int ROUTE_WAVES = 4;      // tokens of a workgroup, one wave each

__device__ __forceinline__ float route_logit(const RouteArgs& a, size_t i) {
    if (a.dtype == W4A8_F32) return static_cast<const float*>(a.logits)[i];
    const uint16_t b = static_cast<const uint16_t*>(a.logits)[i];
    return a.dtype == W4A8_F16 ? f16_to_f32(b) : bf16_to_f32(b);
}

// One wave per token; lane l holds the experts l, l + 64, ... (EPL of them).  Ranks are float64 throughout: a logit is
// exact in it, and p + bias is compared where its last float32 digit would already decide between two experts.
template <int EPL>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void moe_route_kernel(RouteArgs a) {
    extern __shared__ double route_lds[];                       // per wave: ranks [E], scores [E]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x * ROUTE_WAVES + wave;
    if (t >= a.T) return;                                       // no barrier below: waves work alone
    double* lrank = route_lds + size_t(wave) * 2 * a.E;
    double* lp = lrank + a.E;
    const double NEG = -__builtin_huge_val();

    float x[EPL];
    double rank[EPL], p[EPL];
    bool bad = false;
    float top = -__builtin_huge_valf();
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = j * 64 + lane;
        x[j] = e < a.E ? route_logit(a, size_t(t) * a.ldl + e) : -__builtin_huge_valf();
        bad |= x[j] != x[j] || (!a.sigmoid && x[j] == __builtin_huge_valf());
        top = fmaxf(top, x[j]);
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const bool masked = x[j] == -__builtin_huge_valf();
        p[j] = masked ? 0.0 : a.sigmoid ? 1.0 / (1.0 + exp(-double(x[j]))) : exp(double(x[j]) - double(top));
        sum += p[j];
    }
    if (!a.sigmoid) {
#pragma unroll
        for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o, 64);
#pragma unroll
        for (int j = 0; j < EPL; ++j) p[j] = sum > 0.0 ? p[j] / sum : 0.0;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = j * 64 + lane;
        const bool masked = x[j] == -__builtin_huge_valf();
        rank[j] = masked ? NEG : a.bias ? p[j] + double(a.bias[e]) : double(x[j]);
        bad |= rank[j] != rank[j];
        if (e < a.E) {
            lrank[e] = rank[j];
            lp[e] = p[j];
        }
    }
    bad = __any(bad);
    __builtin_amdgcn_wave_barrier();
    if (a.groups > 1 && !bad) {
        // lane g scores the groups g, g + 64, ...; then the `keep` best by repeated choice
        const int size = a.E / a.groups;
        unsigned kept = 0;                                      // bit i: group 64 i + lane is kept
        double best[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int g = i * 64 + lane;
            best[i] = NEG;
            if (i * 64 >= a.groups) continue;
            double b1 = NEG, b2 = NEG;
            if (g < a.groups)
                for (int m = 0; m < size; ++m) {
                    const double r = lrank[g * size + m];
                    if (r > b1) b2 = b1, b1 = r;
                    else if (r > b2) b2 = r;
                }
            best[i] = a.bias && b2 != NEG ? b1 + b2 : b1;
        }
        for (int r = 0; r < a.keep; ++r) {
            double m = NEG;
            int mg = 0x7fffffff;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i * 64 < a.groups && !((kept >> i) & 1) && best[i] > m) m = best[i], mg = i * 64 + lane;
#pragma unroll
            for (int o = 32; o; o >>= 1) {
                const double om = __shfl_xor(m, o, 64);
                const int og = __shfl_xor(mg, o, 64);
                if (om > m || (om == m && og < mg)) m = om, mg = og;
            }
            if (mg == 0x7fffffff) break;                        // no group with a free expert is left
            if ((mg & 63) == lane) kept |= 1u << (mg >> 6);
        }
        // every expert asks the lane that holds its group
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = j * 64 + lane, g = e < a.E ? e / size : 0;
            const unsigned bits = unsigned(__shfl(int(kept), g & 63, 64));
            if (!((bits >> (g >> 6)) & 1)) rank[j] = NEG;
        }
    }
    int id = -1;
    for (int r = 0; r < a.k; ++r) {
        double m = NEG;
        int me = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (rank[j] > m) m = rank[j], me = j * 64 + lane;
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            const double om = __shfl_xor(m, o, 64);
            const int oe = __shfl_xor(me, o, 64);
            if (om > m || (om == m && oe < me)) m = om, me = oe;
        }
        if (me == 0x7fffffff) break;
        if (lane == r) id = me;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (j * 64 + lane == me) rank[j] = NEG;
    }
    double w = id >= 0 ? lp[id] : 0.0;
    if (a.renorm) {
        double s = lane < a.k ? w : 0.0;
#pragma unroll
        for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o, 64);
        w = s > 0.0 ? w / s : 0.0;
    }
    if (lane < a.k) {
        a.ids[size_t(t) * a.k + lane] = bad ? lane : id;
        a.w[size_t(t) * a.k + lane] = bad ? __builtin_nanf("") : float(w * double(a.scale));
    }
}

}  // namespace w4a8

using namespace w4a8;

extern "C" int w4a8_moe_route(const void* logits, int dtype, int T, int ldl, const float* bias, const w4a8_route_desc* d,
                              int32_t* ids, float* w, void* stream) {
    if (!d || T < 0 || d->E <= 0 || d->k <= 0 || d->k > d->E || ldl < d->E) return W4A8_EINVAL;
    if (dtype != W4A8_BF16 && dtype != W4A8_F32 && dtype != W4A8_F16) return W4A8_EINVAL;
    if (d->score != W4A8_ROUTE_SOFTMAX && d->score != W4A8_ROUTE_SIGMOID) return W4A8_EINVAL;
    if (d->renormalize != 0 && d->renormalize != 1) return W4A8_EINVAL;
    const int groups = d->n_group <= 1 ? 1 : d->n_group, keep = groups == 1 ? 1 : d->topk_group;
    if (d->n_group < 0 || d->E % groups || keep < 1 || keep > groups || keep * (d->E / groups) < d->k) return W4A8_EINVAL;
    if (!(std::fabs(d->scale) <= 3.40282347e38f)) return W4A8_EINVAL;
    if (d->E > 1024 || d->k > 64 || T > (1 << 24)) return W4A8_EUNSUPPORTED;
    if (T == 0) return W4A8_OK;
    if (!logits || !ids || !w) return W4A8_EINVAL;
    if (reinterpret_cast<uintptr_t>(logits) & (dtype == W4A8_F32 ? 3u : 1u)) return W4A8_EINVAL;
    if ((reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(bias)) & 3u)
        return W4A8_EINVAL;
    const RouteArgs a{logits, dtype, T, ldl, bias, d->E, d->k, d->score == W4A8_ROUTE_SIGMOID, d->renormalize, groups, keep,
                      d->scale, ids, w};
    const dim3 grid((T + ROUTE_WAVES - 1) / ROUTE_WAVES), block(64 * ROUTE_WAVES);
    const size_t lds = size_t(ROUTE_WAVES) * 2 * d->E * sizeof(double);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (d->E <= 64) moe_route_kernel<1><<<grid, block, lds, s>>>(a);
    else if (d->E <= 128) moe_route_kernel<2><<<grid, block, lds, s>>>(a);
    else if (d->E <= 256) moe_route_kernel<4><<<grid, block, lds, s>>>(a);
    else if (d->E <= 512) moe_route_kernel<8><<<grid, block, lds, s>>>(a);
    else moe_route_kernel<16><<<grid, block, lds, s>>>(a);
    return hipGetLastError() == hipSuccess ? W4A8_OK : W4A8_EHIP;
}
