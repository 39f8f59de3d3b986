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
    int E, k, sigmoid, renorm, groups, keep, gsize;
    float scale;
    int32_t* ids;
    float* w;
};

constexpr int ROUTE_WAVES = 4;      // waves of a workgroup

__device__ __forceinline__ float route_logit(const RouteArgs& a, size_t i) {
    if (a.dtype == W4A8_F32) return static_cast<const float*>(a.logits)[i];
    const uint16_t b = static_cast<const uint16_t*>(a.logits)[i];
    return a.dtype == W4A8_F16 ? f16_to_f32(b) : bf16_to_f32(b);
}

// exp(y) for |y| <= 750, relative error below 2^-50 near 0 and 2^-45 at the ends: y = n ln 2 + r with |r| <= 0.35, where
// n is what adding 1.5 2^52 leaves in the low bits; exp(r) = 1 + r q(r) with q the polynomial that meets it at the 10
// Chebyshev nodes of that range (the Taylor series needs two terms more); scaled by 2^n.
__device__ __forceinline__ double route_exp(double y) {
    const double t = fma(y, 1.4426950408889634, 6755399441055744.0), n = t - 6755399441055744.0;
    const double r = fma(n, -0.6931471805599453, y);
    double e = 0x1.289185613a3d6p-22;
    e = fma(e, r, 0x1.72e1150d0c9b6p-19);
    e = fma(e, r, 0x1.a019b90d2ae7ap-16);
    e = fma(e, r, 0x1.a01994bd214e7p-13);
    e = fma(e, r, 0x1.6c16c1788bd90p-10);
    e = fma(e, r, 0x1.11111123c1f47p-7);
    e = fma(e, r, 0x1.5555555553d63p-5);
    e = fma(e, r, 0x1.5555555550d79p-3);
    e = fma(e, r, 0x1.0000000000001p-1);
    e = fma(e, r, 1.0);
    e = fma(e, r, 1.0);
    return ldexp(e, int(uint32_t(__builtin_bit_cast(uint64_t, t))));
}
__device__ __forceinline__ double exp_neg(double a) { return route_exp(-fmin(a, 750.0)); }   // a >= 0; exp(-750) is 0

// 1 / d for 1 <= d <= 2^1022: the hardware's estimate (2^-23) and one step of third order.
__device__ __forceinline__ double reciprocal(double d) {
    const double r = __builtin_amdgcn_rcp(d), u = fma(-d, r, 1.0);
    return fma(fma(u, u, u), r, r);
}

__device__ __forceinline__ double sigmoid64(float x) {
    const double e = exp_neg(fabs(double(x))), d = reciprocal(1.0 + e);
    return x >= 0.0f ? d : e * d;
}

// The same for a rank: one form for both signs, in which logits below -708 count as -708 (a score of 3e-308).
__device__ __forceinline__ double sigmoid_rank(float x) {
    return reciprocal(1.0 + route_exp(double(__builtin_amdgcn_fmed3f(-x, -745.0f, 708.0f))));
}

// exp(-a) for a >= 0 in float32, good to about 2 units: v_exp_f32 of the product in two parts.
__device__ __forceinline__ float exp_neg32(float a) {
    a = fminf(a, 200.0f);                                       // exp(-200) is 0 in float32
    const float t = -a * 1.44269502f, r = fmaf(-a, 1.44269502f, -t) - a * 1.92596303e-8f;
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, r * 0.693147182f, e);
}

// A rank as a sorting key: the float64 value with its last 10 mantissa bits replaced by the index, turned so that of two
// equal values the lower index is the larger key (of a negative value the larger mantissa is the smaller number).  One
// v_max_f64 then compares value and index.  Logits are float32 and lose nothing; p + bias, and the sum of two of them that ranks a group, keep 42 bits.
constexpr double ROUTE_NONE = -1.7e308;                         // a masked or taken expert; ranks are above -1e39

__device__ __forceinline__ double route_key(double v, int index) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t sign = uint32_t(int32_t(b >> 32) >> 31), low = sign ^ uint32_t(index ^ 1023);
    return __builtin_bit_cast(double, (b & ~uint64_t(1023)) | (low & 1023u));
}
__device__ __forceinline__ int route_index(double key) {
    const uint64_t b = __builtin_bit_cast(uint64_t, key);
    return int((uint32_t(b) ^ ~uint32_t(int32_t(b >> 32) >> 31)) & 1023u);
}
// the key of a masked expert: a number below all ranks, whatever its low half
__device__ __forceinline__ double route_mask(double key, bool masked) {
    const uint64_t b = __builtin_bit_cast(uint64_t, key);
    const uint32_t hi = masked ? uint32_t(__builtin_bit_cast(uint64_t, ROUTE_NONE) >> 32) : uint32_t(b >> 32);
    return __builtin_bit_cast(double, uint64_t(hi) << 32 | uint32_t(b));
}
__device__ __forceinline__ double route_value(double key) {
    return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, key) & ~uint64_t(1023));
}

// What the lane across from this one holds: STEP 0..3 exchange neighbours, pairs, quads and halves of 16 lanes (the last two
// by mirroring, which is the same thing once the smaller groups agree), STEP 4 the 16s of 32 and STEP 5 the halves of 64.
template <int STEP>
__device__ __forceinline__ uint32_t route_across(uint32_t v) {
    if constexpr (STEP == 0) return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xF, 0xF, true));
    else if constexpr (STEP == 1) return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4E, 0xF, 0xF, true));
    else if constexpr (STEP == 2) return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x141, 0xF, 0xF, true));
    else if constexpr (STEP == 3) return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x140, 0xF, 0xF, true));
    else return uint32_t(__shfl_xor(int(v), STEP == 4 ? 16 : 32, 64));
}
template <int STEP>
__device__ __forceinline__ double route_across(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = route_across<STEP>(uint32_t(b)), hi = route_across<STEP>(uint32_t(b >> 32));
    return __builtin_bit_cast(double, hi << 32 | lo);
}
template <int STEP>
__device__ __forceinline__ float route_across(float v) {
    return __uint_as_float(route_across<STEP>(__float_as_uint(v)));
}
// v combined over the LANES lanes of a token, the same in all of them and in a fixed order
template <int LANES, typename T, typename F>
__device__ __forceinline__ T route_all(T v, F f) {
    v = f(v, route_across<0>(v));
    v = f(v, route_across<1>(v));
    v = f(v, route_across<2>(v));
    v = f(v, route_across<3>(v));
    if constexpr (LANES > 16) v = f(v, route_across<4>(v));
    if constexpr (LANES > 32) v = f(v, route_across<5>(v));
    return v;
}

// Descending order of key[LO .. LO + N): Batcher's odd-even merge sort, unrolled; what no one reads of its end is left out
// by the compiler.
template <int LO, int N, int STEP, int EPL>
__device__ __forceinline__ void route_merge(double (&key)[EPL]) {
    const auto swap = [&](int i, int j) __attribute__((always_inline)) {
        const double u = key[i], v = key[j];
        key[i] = fmax(u, v), key[j] = fmin(u, v);
    };
    if constexpr (2 * STEP < N) {
        route_merge<LO, N, 2 * STEP>(key);
        route_merge<LO + STEP, N, 2 * STEP>(key);
#pragma unroll
        for (int i = STEP; i + STEP < N; i += 2 * STEP) swap(LO + i, LO + i + STEP);
    } else {
        swap(LO, LO + STEP);
    }
}
template <int LO, int N, int EPL>
__device__ __forceinline__ void route_sort(double (&key)[EPL]) {
    if constexpr (N > 1) {
        route_sort<LO, N / 2>(key);
        route_sort<LO + N / 2, N / 2>(key);
        route_merge<LO, N, 1>(key);
    }
}

// LANES lanes per token, EPL neighbouring experts in each, of which a lane keeps the DEPTH >= min(k, EPL) best in order;
// k <= LANES rounds, each the best of the lanes' first keys, which its lane then drops.  A group of experts, or all of
// them, has 2^gshift whole lanes, of which the last may be filled in part or not at all.  With 16 lanes a wave serves 4 tokens.  The vector unit is the bound of many tokens: 16384
// of 256 experts with bias and groups take 1273 instructions a wave, 8.5 of the kernel's 12.5 us (a search of all keys in
// each round and the Taylor series: 1949 and 18.0 us); half of them are the float64 scores and the keys.
template <int LANES, int EPL, int DEPTH>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void moe_route_kernel(RouteArgs a, int gshift) {
    constexpr int TOKENS = 64 / LANES * ROUTE_WAVES;
    const int lane = threadIdx.x % LANES, group = lane >> gshift, first = (lane - (group << gshift)) * EPL;
    const int e0 = group * a.gsize + first, count = group < a.groups ? min(a.gsize - first, EPL) : 0;
    const int t0 = int(blockIdx.x) * TOKENS + int(threadIdx.x) / LANES;
    const int t = min(t0, a.T - 1);                             // every lane takes part in the exchanges
    const size_t row = size_t(t) * size_t(a.ldl);
    const auto max64 = [](double x, double y) { return fmax(x, y); };

    float x[EPL];
    const bool full = count == EPL && (e0 & 3) == 0;            // whole and aligned vectors
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.logits);
    if (a.dtype == W4A8_F32 && full && !(base & 15) && !(a.ldl & 3)) {
#pragma unroll
        for (int j = 0; j < EPL; j += 4) {
            const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + row + e0 + j);
            x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
        }
    } else if (a.dtype != W4A8_F32 && full && !(base & 7) && !(a.ldl & 3)) {
#pragma unroll
        for (int j = 0; j < EPL; j += 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + row + e0 + j);
            const uint32_t h[4] = {v.x & 0xffffu, v.x >> 16, v.y & 0xffffu, v.y >> 16};
#pragma unroll
            for (int i = 0; i < 4; ++i) x[j + i] = a.dtype == W4A8_F16 ? f16_to_f32(uint16_t(h[i])) : bf16_to_f32(h[i]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) x[j] = j < count ? route_logit(a, row + e0 + j) : -__builtin_huge_valf();
    }
    bool bad = false;
    float top = -__builtin_huge_valf();
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        bad |= x[j] != x[j] || (!a.sigmoid && x[j] == __builtin_huge_valf());
        top = fmaxf(top, x[j]);
    }
    const auto max32 = [](float u, float v) { return fmaxf(u, v); };
    double key[EPL], sum = 1.0;                                 // sum: softmax denominator
    if (!a.sigmoid) top = route_all<LANES>(top, max32);
    const float ref = top > -__builtin_huge_valf() ? top : 0.0f;
    if (a.bias) {
        double p[EPL];
        float bias[EPL];
        if (full && !(reinterpret_cast<uintptr_t>(a.bias) & 15)) {
#pragma unroll
            for (int j = 0; j < EPL; j += 4) {
                const float4 v = *reinterpret_cast<const float4*>(a.bias + e0 + j);
                bias[j] = v.x, bias[j + 1] = v.y, bias[j + 2] = v.z, bias[j + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j) bias[j] = j < count ? a.bias[e0 + j] : 0.0f;
        }
        if (a.sigmoid) {
#pragma unroll
            for (int j = 0; j < EPL; ++j) p[j] = sigmoid_rank(x[j]);
        } else {
            sum = 0.0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                p[j] = exp_neg(double(ref) - double(x[j]));
                sum += p[j];
            }
            sum = route_all<LANES>(sum, [](double u, double v) { return u + v; });
            const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) p[j] *= inv;
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            // a masked expert ranks as one with a bias of -Inf, whatever its own is
            const double r = p[j] + double(x[j] == -__builtin_huge_valf() ? x[j] : bias[j]);
            bad |= r != r;
            // an infinite bias stays a number
            key[j] = route_mask(route_key(fmin(r, 1e300), e0 + j), r < -1e39);
        }
    } else {
        if (!a.sigmoid) {
            float part = 0.0f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) part += exp_neg32(ref - x[j]);
            sum = double(route_all<LANES>(part, [](float u, float v) { return u + v; }));
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j)                           // -0 equals 0; an infinity stays a number
            key[j] = route_mask(route_key(fmin(double(x[j]) + 0.0, 1e300), e0 + j), x[j] == -__builtin_huge_valf());
    }
    bad = route_all<LANES>(uint32_t(bad), [](uint32_t u, uint32_t v) { return u | v; }) != 0;
    if constexpr (DEPTH == EPL) {
        route_sort<0, EPL>(key);
    } else {                                                    // the better half of two sorted halves, then sorted itself
        route_sort<0, DEPTH>(key);
        route_sort<DEPTH, DEPTH>(key);
#pragma unroll
        for (int j = 0; j < DEPTH; ++j) key[j] = fmax(key[j], key[EPL - 1 - j]);
#pragma unroll
        for (int d = DEPTH / 2; d; d /= 2)
#pragma unroll
            for (int j = 0; j < DEPTH; ++j)
                if (!(j & d)) {
                    const double u = key[j], v = key[j + d];
                    key[j] = fmax(u, v), key[j + d] = fmin(u, v);
                }
    }

    if (a.groups > 1) {
        double b1 = key[0], b2 = key[1];                        // the group's two best
        auto merge = [&](double c1, double c2) __attribute__((always_inline)) {
            b2 = fmax(fmax(b2, c2), fmin(b1, c1));
            b1 = fmax(b1, c1);
        };
        if (gshift > 0) merge(route_across<0>(b1), route_across<0>(b2));
        if (gshift > 1) merge(route_across<1>(b1), route_across<1>(b2));
        if (gshift > 2) merge(route_across<2>(b1), route_across<2>(b2));
        if (gshift > 3) merge(route_across<3>(b1), route_across<3>(b2));
        if (gshift > 4) merge(route_across<4>(b1), route_across<4>(b2));
        double score = ROUTE_NONE;
        if (b1 > -1e300 && group < a.groups)
            score = route_key(fmin(a.bias && b2 > -1e300 ? route_value(b1) + route_value(b2) : route_value(b1), 1e300), group);
        bool kept = false;
        for (int r = 0; r < a.keep; ++r) {
            const double best = route_all<LANES>(score, max64);
            if (best > -1e300 && score == best) kept = true, score = ROUTE_NONE;
        }
#pragma unroll
        for (int j = 0; j < DEPTH; ++j) key[j] = route_mask(key[j], !kept);
    }

    int id = -1;                                                // of round `lane`
    for (int r = 0; r < a.k; ++r) {
        const double best = route_all<LANES>(key[0], max64);
        if (lane == r && best > -1e300) id = route_index(best);
        const bool mine = key[0] == best;
#pragma unroll
        for (int j = 0; j < DEPTH - 1; ++j) key[j] = mine ? key[j + 1] : key[j];
        key[DEPTH - 1] = route_mask(key[DEPTH - 1], mine);
    }
    double w = 0.0;
    if (id >= 0) {
        const float v = route_logit(a, row + id);
        w = a.sigmoid ? sigmoid64(v) : exp_neg(double(ref) - double(v)) / sum;
    }
    if (a.renorm) {
        const double s = route_all<LANES>(w, [](double u, double v) { return u + v; });
        w = s > 0.0 ? w / s : 0.0;
    }
    if (lane < a.k && t0 < a.T) {
        a.ids[size_t(t) * a.k + lane] = bad ? lane : id;
        a.w[size_t(t) * a.k + lane] = bad ? __builtin_nanf("") : float(w * double(a.scale));
    }
}

// More groups than the kernel above has lanes for (100 groups of 2, 3 of 340): one wave per token, the ranks in LDS for the
// group scores.
// Lane l holds the experts l, l + 64, ... (EPL of them); ranks as above.
template <int EPL>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void moe_route_any_groups_kernel(RouteArgs a) {
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
        p[j] = masked ? 0.0 : a.sigmoid ? sigmoid64(x[j]) : exp_neg(double(top) - double(x[j]));
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
        rank[j] = masked ? NEG : a.bias ? (e < a.E ? p[j] + double(a.bias[e]) : 0.0) : double(x[j]);
        bad |= rank[j] != rank[j];
        if (!masked && a.bias) rank[j] = rank[j] < -1e39 ? NEG : route_value(rank[j]);
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
            best[i] = a.bias && b2 != NEG ? route_value(b1 + b2) : b1;
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
                      d->E / groups, d->scale, ids, w};
    hipStream_t s = static_cast<hipStream_t>(stream);
    // The first form that holds a token.  64 lanes only where the rounds or the experts need more than 16: those are no
    // slower for few tokens either (64 tokens of 256 experts 5.2 against 5.3 us, of 64 experts 2.8 against 4.1) and faster
    // for many (4096: 5.6 against 8.1).
    constexpr struct { int lanes, epl; } forms[] = {{16, 4}, {16, 8}, {16, 16}, {64, 4}, {64, 16}};
    int form = 0, gshift = 0;
    for (; form < 5; ++form) {
        gshift = 0;
        while ((forms[form].epl << gshift) < a.gsize) ++gshift;
        if (d->k <= forms[form].lanes && (groups << gshift) <= forms[form].lanes) break;
    }
    const int tokens = ROUTE_WAVES * (form < 3 ? 4 : 1);
    const dim3 grid((T + tokens - 1) / tokens), block(64 * ROUTE_WAVES);
    if (form == 0) moe_route_kernel<16, 4, 4><<<grid, block, 0, s>>>(a, gshift);
    else if (form == 1) moe_route_kernel<16, 8, 8><<<grid, block, 0, s>>>(a, gshift);
    else if (form == 2 && d->k <= 8) moe_route_kernel<16, 16, 8><<<grid, block, 0, s>>>(a, gshift);
    else if (form == 2) moe_route_kernel<16, 16, 16><<<grid, block, 0, s>>>(a, gshift);
    else if (form == 3) moe_route_kernel<64, 4, 4><<<grid, block, 0, s>>>(a, gshift);
    else if (form == 4) moe_route_kernel<64, 16, 16><<<grid, block, 0, s>>>(a, gshift);
    else {
        const size_t lds = size_t(ROUTE_WAVES) * 2 * d->E * sizeof(double);
        if (d->E <= 256) moe_route_any_groups_kernel<4><<<grid, block, lds, s>>>(a);
        else moe_route_any_groups_kernel<16><<<grid, block, lds, s>>>(a);
    }
    return hipGetLastError() == hipSuccess ? W4A8_OK : W4A8_EHIP;
}
