// Microscaled (MX) formats: blocks of 32 neighbours along K share one power-of-two scale.  Layouts, the block rule and the
// element conversions shared by the MX kernels (gfx950).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "w4a8_internal.h"
#include "w4a8_device.h"

namespace w4a8 {

typedef float v2f __attribute__((ext_vector_type(2)));
typedef int v2i __attribute__((ext_vector_type(2)));

// K of a stored row: padded with zeros to whole MFMA steps of 128.
constexpr int MX_STEP = 128;
inline __host__ __device__ int mx_kp(int K) { return (K + MX_STEP - 1) / MX_STEP * MX_STEP; }
inline __host__ __device__ size_t mx_row_bytes(int fmt, int K) { return size_t(mx_kp(K)) / (fmt == W4A8_MX_FP4 ? 2 : 1); }

// Limits of the MX calls: 32-bit offsets within a row and within a call's tiles.
constexpr int MX_MAX_K = 1 << 20;
constexpr int MX_MAX_N = 1 << 20;
int mx_check_weights(int N, int K);                             // OK, EINVAL or EUNSUPPORTED

// Packed fp4 weights [N, K]: codes by 16 columns x 128 k (1 KiB, the order of an MFMA operand), then scales by 64 columns x
// 128 k (256 bytes: lane l of a wave finds those of the four 16-column operands in one word).
struct MxLayout {
    int K1;                                                     // steps of 128 k
    size_t codes_bytes, scales_off, scales_bytes, total;
};
inline __host__ __device__ MxLayout mx_layout(int N, int K) {
    MxLayout L;
    L.K1 = mx_kp(K) / MX_STEP;
    L.codes_bytes = size_t((N + 15) / 16) * size_t(L.K1) * 1024;
    L.scales_off = (L.codes_bytes + 255) & ~size_t(255);
    L.scales_bytes = size_t((N + 63) / 64) * size_t(L.K1) * 256;
    L.total = L.scales_off + L.scales_bytes;
    return L;
}

// Scale byte of a block whose largest magnitude has the bit pattern amax: the power of two under it, less the format's largest
// exponent (2 for E2M1, 8 for E4M3), not below 2^-127.  255 (NaN) if the block holds a NaN or an infinity.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
    const int b = int(amax >> 23) - (FMT == W4A8_MX_FP4 ? 2 : 8);
    return amax >= 0x7f800000u ? 255u : uint32_t(max(b, 0));
}

// 2^(127 - b), what the elements of a block are multiplied by: a normal number for every b of a finite block (b <= 252).
__device__ __forceinline__ float mx_up(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// 2^(b - 127): 2^-127 is not a normal number, 255 is NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255u ? 0x7fc00000u : b << 23);
}

// Four elements x / scale, to nearest even, saturating at the largest element.  v_cvt_scalef32_pk_fp4_f32 saturates by itself;
// v_cvt_pk_fp8_f32 makes a NaN of what is past 448, so that is clamped first.
__device__ __forceinline__ uint32_t mx_fp4x4(const float x0, const float x1, const float x2, const float x3) {
    uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x0, x1, 1.0f, 0);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x2, x3, 1.0f, 1) & 0xffffu;
}
__device__ __forceinline__ uint32_t mx_fp8x4(const float x0, const float x1, const float x2, const float x3) {
    auto c = [](float x) __attribute__((always_inline)) { return __builtin_amdgcn_fmed3f(x, -448.0f, 448.0f); };
    const int r = __builtin_amdgcn_cvt_pk_fp8_f32(c(x0), c(x1), 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c(x2), c(x3), r, true));
}

// Largest magnitude's bits of 8 values.  As integers: a NaN counts above everything.
__device__ __forceinline__ uint32_t mx_amax8(const float* v) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

// Maximum over the 4 neighbouring lanes that hold a block (quad permutes by 1 and by 2).
__device__ __forceinline__ uint32_t mx_quad_max(uint32_t m) {
    m = max(m, uint32_t(__builtin_amdgcn_mov_dpp(int(m), 0xB1, 0xF, 0xF, true)));
    return max(m, uint32_t(__builtin_amdgcn_mov_dpp(int(m), 0x4E, 0xF, 0xF, true)));
}

// f over all 64 lanes, in every lane: exchanges within rows of 16 by DPP (quad permutes, half and whole row mirrored), between
// rows by v_permlane{16,32}_swap; no LDS.
template <class F>
__device__ __forceinline__ uint32_t wave_all(uint32_t m, F f) {
    m = f(m, uint32_t(__builtin_amdgcn_mov_dpp(int(m), 0xB1, 0xF, 0xF, true)));
    m = f(m, uint32_t(__builtin_amdgcn_mov_dpp(int(m), 0x4E, 0xF, 0xF, true)));
    m = f(m, uint32_t(__builtin_amdgcn_mov_dpp(int(m), 0x141, 0xF, 0xF, true)));
    m = f(m, uint32_t(__builtin_amdgcn_mov_dpp(int(m), 0x140, 0xF, 0xF, true)));
    const auto a = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = f(uint32_t(a[0]), uint32_t(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return f(uint32_t(b[0]), uint32_t(b[1]));
}
__device__ __forceinline__ float wave_sum(float s) {
    return __uint_as_float(wave_all(__float_as_uint(s), [](uint32_t x, uint32_t y) __attribute__((always_inline)) {
        return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
    }));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
    return wave_all(m, [](uint32_t x, uint32_t y) __attribute__((always_inline)) { return max(x, y); });
}

// 8 neighbouring elements at p, of which n exist (the others are 0), as float32.  Any alignment of whole elements.
template <int DT>
__device__ __forceinline__ void mx_load8(const void* p, const int n, float* v) {
    if constexpr (DT == W4A8_F32) {
        typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
        const float* x = static_cast<const float*>(p);
        if (n >= 8) {
            const f4 a = *reinterpret_cast<const f4*>(x), b = *reinterpret_cast<const f4*>(x + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? x[i] : 0.0f;
        }
    } else {
        typedef uint16_t u8x __attribute__((ext_vector_type(8), aligned(2)));
        const uint16_t* x = static_cast<const uint16_t*>(p);
        u8x a = {0, 0, 0, 0, 0, 0, 0, 0};
        if (n >= 8) {
            a = *reinterpret_cast<const u8x*>(x);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) a[i] = x[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = DT == W4A8_F16 ? f16_to_f32(a[i]) : bf16_to_f32(a[i]);
    }
}

// Stores 8 neighbouring elements at p, of which n exist, rounded to nearest even.
template <int DT>
__device__ __forceinline__ void mx_store8(void* p, const int n, const float* v) {
    if constexpr (DT == W4A8_F32) {
        typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
        float* y = static_cast<float*>(p);
        if (n >= 8) {
            *reinterpret_cast<f4*>(y) = f4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f4*>(y + 4) = f4{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) y[i] = v[i];
        }
    } else {
        typedef uint16_t u8x __attribute__((ext_vector_type(8), aligned(2)));
        uint16_t* y = static_cast<uint16_t*>(p);
        u8x a;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            a[i] = DT == W4A8_F16 ? __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[i])) : uint16_t(f32_to_bf16_rne(v[i]));
        if (n >= 8) {
            *reinterpret_cast<u8x*>(y) = a;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) y[i] = a[i];
        }
    }
}

// 8 values of one block, whose largest magnitude's bits over all 32 are amax, as elements: 4 (fp4) or 8 bytes.
template <int FMT>
__device__ __forceinline__ uint2 mx_encode8(const float* v, const uint32_t byte) {
    if (byte == 255u) return make_uint2(0u, 0u);
    const float up = mx_up(byte);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = v[i] * up;
    if constexpr (FMT == W4A8_MX_FP4)
        return make_uint2(mx_fp4x4(y[0], y[1], y[2], y[3]) | (mx_fp4x4(y[4], y[5], y[6], y[7]) << 16), 0u);
    else
        return make_uint2(mx_fp8x4(y[0], y[1], y[2], y[3]), mx_fp8x4(y[4], y[5], y[6], y[7]));
}

}  // namespace w4a8
