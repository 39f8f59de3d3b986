// The norm around a block: RMS norm, gate and scale of the block's output, the sum into the residual stream, and the RMS norm in
// front of the next block with its activation quantisation, in one pass over the rows.
//
// Sources (cited with the page's own section names):
//   P2 "Kimi 2.7 MoE W4A8: 4-bit storage to INT8, deployment notes" (xdnf.cn), section 3.3: a quantize node before each Linear.
//   P3 "Quantization: formats, error and the real execution path" (wineandchord.com), "Weight-Activation": scalings fused into
//      an adjacent operator.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>

#include "w4a8_mx.h"

namespace w4a8 {

struct NormArgs {
    const uint8_t* X;
    const uint8_t* res;       // NULL: zeros
    const uint8_t* gate;      // NULL: ones
    const float* post_w;      // NULL: no norm of X
    const float* w;
    uint8_t* res_out;         // NULL: not stored
    uint8_t* Y;               // h, or its codes
    uint8_t* sx;
    long long ldx, ldr, ldg, ldo, ldy;
    int M, H, fmt;
    float eps, eps_post, alpha;
};

enum { NORM_NONE = -1, NORM_H = -2 };                           // beside the formats of quantised h

// v as the type that it is stored in.
template <int DT>
__device__ __forceinline__ float round_to(float v) {
    if constexpr (DT == W4A8_F32) return v;
    else if constexpr (DT == W4A8_F16) return static_cast<float>(static_cast<_Float16>(v));
    else return bf16_to_f32(f32_to_bf16_rne(v));
}

// WPR waves hold a row in registers, 8 neighbours a lane in each of R rounds, so that everything is read once and written once.
// Sums of squares: each lane's, then across the wave, then (WPR > 1) across the waves through LDS, all in float32 and in a
// fixed order.  Bound by the copy: 8192 rows of 7168 with a float32 residual stream and a gate for each token (822 MB) take 160 us,
// 5.1 TB/s, the rate of a large copy.
template <int DT, int RT, int WPR, int R>
__global__ __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) void norm_residual_kernel(NormArgs a) {
    constexpr int ES = DT == W4A8_F32 ? 4 : 2, RS = RT == W4A8_F32 ? 4 : 2, T = 64 * WPR;
    __shared__ float part[3][16];
    const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
    const int row = WPR == 1 ? int(blockIdx.x) * 4 + wave : int(blockIdx.x);
    const int t = WPR == 1 ? lane : int(threadIdx.x);
    if (WPR == 1 && row >= a.M) return;
    const int Kp = mx_kp(a.H);

    auto sum = [&](float s, const int which) __attribute__((always_inline)) {
        s = wave_sum(s);
        if constexpr (WPR > 1) {
            if (lane == 0) part[which][wave] = s;
            __syncthreads();
            s = part[which][0];
#pragma unroll
            for (int w = 1; w < WPR; ++w) s += part[which][w];
        }
        return s;
    };
    // few values a lane: the weights are requested with everything else, and not after the sums that they wait for
    constexpr bool EARLY = R <= 2;
    float w[EARLY ? R : 1][8], p[EARLY ? R : 1][8], g[EARLY ? R : 1][8];

    float v[R][8], r[R][8];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int k = (i * T + t) * 8, n = a.H - k;
        mx_load8<DT>(a.X + (size_t(row) * size_t(a.ldx) + size_t(min(k, a.H))) * ES, n, v[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int k = (i * T + t) * 8, n = a.H - k;
        if (a.res) {
            mx_load8<RT>(a.res + (size_t(row) * size_t(a.ldr) + size_t(min(k, a.H))) * RS, n, r[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] = 0.0f;
        }
    }
    if constexpr (EARLY) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int k = (i * T + t) * 8, n = a.H - k;
            if (a.gate) mx_load8<DT>(a.gate + (size_t(row) * size_t(a.ldg) + size_t(min(k, a.H))) * ES, n, g[i]);
            if (a.post_w) mx_load8<W4A8_F32>(a.post_w + min(k, a.H), n, p[i]);
            if (a.fmt != NORM_NONE) mx_load8<W4A8_F32>(a.w + min(k, a.H), n, w[i]);
        }
    }
    if (a.post_w) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(v[i][j], v[i][j], s);
        const float rs = 1.0f / sqrtf(sum(s, 0) / float(a.H) + a.eps_post);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int k = (i * T + t) * 8, n = a.H - k;
            const int at = EARLY ? i : 0;
            if (!EARLY) mx_load8<W4A8_F32>(a.post_w + min(k, a.H), n, p[at]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rs * p[at][j];
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int k = (i * T + t) * 8, n = a.H - k;
        if (a.gate) {
            const int at = EARLY ? i : 0;
            if (!EARLY) mx_load8<DT>(a.gate + (size_t(row) * size_t(a.ldg) + size_t(min(k, a.H))) * ES, n, g[at]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= g[at][j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = round_to<RT>(fmaf(a.alpha, v[i][j], r[i][j]));
        if (a.res_out && n > 0) mx_store8<RT>(a.res_out + (size_t(row) * size_t(a.ldo) + size_t(k)) * RS, n, r[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(r[i][j], r[i][j], s);
    }
    if (a.fmt == NORM_NONE) return;
    const float rs = 1.0f / sqrtf(sum(s, 1) / float(a.H) + a.eps);
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int k = (i * T + t) * 8, n = a.H - k;
        const int at = EARLY ? i : 0;
        if (!EARLY) mx_load8<W4A8_F32>(a.w + min(k, a.H), n, w[at]);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = r[i][j] * rs * w[at][j];
        if (a.fmt == NORM_H) {
            if (n > 0) mx_store8<DT>(a.Y + (size_t(row) * size_t(a.ldy) + size_t(k)) * ES, n, r[i]);
            continue;
        }
        // the codes of h as it would be stored.  Places behind the row hold 0 times the row's factor: cleared, since a row with
        // a NaN would spread it there
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = j < n ? round_to<DT>(r[i][j]) : 0.0f;
        if (a.fmt == W4A8_QUANT_INT8) {
            amax = max(amax, mx_amax8(r[i]));
            continue;
        }
        if (k >= Kp) continue;                                  // whole blocks of 4 lanes
        const size_t block = size_t(row) * size_t(Kp / 32) + k / 32;
        const uint32_t m = mx_quad_max(mx_amax8(r[i]));
        if (a.fmt == W4A8_MX_FP4) {
            const uint32_t byte = mx_scale_byte<W4A8_MX_FP4>(m);
            *reinterpret_cast<uint32_t*>(a.Y + block * 16 + (t & 3) * 4) = mx_encode8<W4A8_MX_FP4>(r[i], byte).x;
            if ((t & 3) == 0) a.sx[block] = uint8_t(byte);
        } else {
            const uint32_t byte = mx_scale_byte<W4A8_MX_FP8>(m);
            *reinterpret_cast<uint2*>(a.Y + block * 32 + (t & 3) * 8) = mx_encode8<W4A8_MX_FP8>(r[i], byte);
            if ((t & 3) == 0) a.sx[block] = uint8_t(byte);
        }
    }
    if (a.fmt != W4A8_QUANT_INT8) return;
    amax = wave_max(amax);
    if constexpr (WPR > 1) {
        if (lane == 0) part[2][wave] = __uint_as_float(amax);
        __syncthreads();
#pragma unroll
        for (int x = 0; x < WPR; ++x) amax = max(amax, __float_as_uint(part[2][x]));
    }
    const RowScale q = row_scale(amax);
    if (t == 0) reinterpret_cast<float*>(a.sx)[row] = q.s;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int k = (i * T + t) * 8;
        if (k >= a.H) continue;                                 // H is a multiple of 16 here
        uint32_t c[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            c[j >> 2] |= (uint32_t(q.finite ? quant_one(r[i][j], q.d, q.inv, q.fast) : 0) & 0xffu) << (8 * (j & 3));
        *reinterpret_cast<uint2*>(a.Y + size_t(row) * size_t(a.H) + k) = make_uint2(c[0], c[1]);
    }
}

template <int DT, int RT>
static void launch_norm(const NormArgs& a, hipStream_t s) {
    const int units = (mx_kp(a.H) + 511) / 512;                 // rounds of one wave
    const unsigned M = unsigned(a.M);
    // few rows: as many waves a row as it has rounds, so that a row is one trip to memory and one sum (8 rows of
    // 4096: 5.4 -> 4.5 us)
    if (units <= 1) norm_residual_kernel<DT, RT, 1, 1><<<dim3((M + 3) / 4), dim3(256), 0, s>>>(a);
    else if (units <= 4) norm_residual_kernel<DT, RT, 4, 1><<<dim3(M), dim3(256), 0, s>>>(a);
    else if (units <= 16 && M <= 512) norm_residual_kernel<DT, RT, 16, 1><<<dim3(M), dim3(1024), 0, s>>>(a);
    else if (units <= 8) norm_residual_kernel<DT, RT, 4, 2><<<dim3(M), dim3(256), 0, s>>>(a);
    else if (units <= 16) norm_residual_kernel<DT, RT, 4, 4><<<dim3(M), dim3(256), 0, s>>>(a);
    else if (units <= 32) norm_residual_kernel<DT, RT, 16, 2><<<dim3(M), dim3(1024), 0, s>>>(a);
    else norm_residual_kernel<DT, RT, 16, 8><<<dim3(M), dim3(1024), 0, s>>>(a);
}

static bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
static bool norm_type(int dt) { return dt == W4A8_BF16 || dt == W4A8_F16 || dt == W4A8_F32; }
static size_t type_size(int dt) { return dt == W4A8_F32 ? 4 : 2; }

constexpr int NORM_MAX_H = 65536, NORM_MAX_ROWS = 1 << 22;      // a row fits 1024 threads

static int run_norm(const void* X, int dtype, int ldx, const void* res, int res_dtype, int ldr, const void* gate, int ldg,
                    const float* post_w, const float* w, const w4a8_norm_desc* d, int M, int H, void* res_out, int ldo, void* Y,
                    int ldy, int fmt, void* sx, hipStream_t s) {
    if (!d || !norm_type(dtype) || !norm_type(res_dtype) || M < 0 || H <= 0) return W4A8_EINVAL;
    if (!(d->eps >= 0.0f) || !(d->eps_post >= 0.0f) || !std::isfinite(d->eps) || !std::isfinite(d->eps_post) || !std::isfinite(d->alpha))
        return W4A8_EINVAL;
    if (ldx < H || (res && ldr < H) || (gate && ldg != 0 && ldg < H) || (res_out && ldo < H) || (fmt == NORM_H && ldy < H))
        return W4A8_EINVAL;
    if (fmt == W4A8_QUANT_INT8 && H % 16) return W4A8_EINVAL;
    if (H > NORM_MAX_H || M > NORM_MAX_ROWS) return W4A8_EUNSUPPORTED;
    if ((long long)M * (H > 8192 ? 1024 : 256) >= (1ll << 32)) return W4A8_EUNSUPPORTED;    // work-items of the launch (see launch_norm)
    if (M == 0) return W4A8_OK;
    if (!X || (fmt == NORM_NONE ? !res_out : !Y || !w) || (fmt >= 0 && !sx)) return W4A8_EINVAL;
    const size_t es = type_size(dtype), rs = type_size(res_dtype);
    if (!aligned_to(X, es) || !aligned_to(gate, es) || !aligned_to(res, rs) || !aligned_to(res_out, rs) || !aligned_to(post_w, 4) ||
        !aligned_to(w, 4) || !aligned_to(sx, 4) || !aligned_to(Y, fmt >= 0 ? 16 : es))
        return W4A8_EINVAL;
    NormArgs a;
    a.X = static_cast<const uint8_t*>(X);
    a.res = static_cast<const uint8_t*>(res);
    a.gate = static_cast<const uint8_t*>(gate);
    a.post_w = post_w;
    a.w = w;
    a.res_out = static_cast<uint8_t*>(res_out);
    a.Y = static_cast<uint8_t*>(Y);
    a.sx = static_cast<uint8_t*>(sx);
    a.ldx = ldx, a.ldr = ldr, a.ldg = ldg, a.ldo = ldo, a.ldy = ldy;
    a.M = M, a.H = H, a.fmt = fmt;
    a.eps = d->eps, a.eps_post = d->eps_post, a.alpha = d->alpha;
    auto by_res = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (res_dtype == W4A8_BF16) launch_norm<DT, W4A8_BF16>(a, s);
        else if (res_dtype == W4A8_F16) launch_norm<DT, W4A8_F16>(a, s);
        else launch_norm<DT, W4A8_F32>(a, s);
    };
    if (dtype == W4A8_BF16) by_res(std::integral_constant<int, W4A8_BF16>{});
    else if (dtype == W4A8_F16) by_res(std::integral_constant<int, W4A8_F16>{});
    else by_res(std::integral_constant<int, W4A8_F32>{});
    return hipGetLastError() == hipSuccess ? W4A8_OK : W4A8_EHIP;
}

}  // namespace w4a8

using namespace w4a8;

extern "C" {

int w4a8_norm_residual(const void* X, int dtype, int ldx, const void* residual, int res_dtype, int ldr, const void* gate, int ldg,
                       const float* post_w, const float* w, const w4a8_norm_desc* d, int M, int H, void* residual_out, int ldo,
                       void* Y, int ldy, void* stream) {
    return run_norm(X, dtype, ldx, residual, res_dtype, ldr, gate, ldg, post_w, w, d, M, H, residual_out, ldo, Y, ldy,
                    Y ? NORM_H : NORM_NONE, nullptr, static_cast<hipStream_t>(stream));
}

int w4a8_norm_residual_quant(const void* X, int dtype, int ldx, const void* residual, int res_dtype, int ldr, const void* gate, int ldg,
                             const float* post_w, const float* w, const w4a8_norm_desc* d, int M, int H, void* residual_out, int ldo,
                             int fmt, void* Xq, void* sx, void* stream) {
    if (fmt != W4A8_MX_FP4 && fmt != W4A8_MX_FP8 && fmt != W4A8_QUANT_INT8) return W4A8_EINVAL;
    return run_norm(X, dtype, ldx, residual, res_dtype, ldr, gate, ldg, post_w, w, d, M, H, residual_out, ldo, Xq, 0, fmt, sx,
                    static_cast<hipStream_t>(stream));
}

}  // extern "C"
