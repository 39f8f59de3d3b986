// Expert-grouped GEMMs on 8-bit per-channel blobs and on 16-bit row-major weights: arguments, formats and the
// row-tile lookup shared by their kernels (gfx950).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "w4a8_device.h"

namespace w4a8 {

// Operand formats.  Every kernel works in bytes along K: an MFMA step takes 64 bytes of a row whatever the format
// (64 int8 values on v_mfma_i32_16x16x64_i8, 32 values of 16 bits on v_mfma_f32_16x16x32_{bf16,f16}), 16 bytes a lane, so
// the tile shapes, the staging and the waits are the same and only the instruction and the epilogue differ.
enum GroupedFormat { GF_I8 = 0, GF_BF16 = 1, GF_F16 = 2 };

struct GroupedArgs {
    const uint8_t* X;         // activation rows
    long long ldx;            // bytes between them
    const float* sx;          // GF_I8: scale of each activation row
    const int32_t* gather;    // source row of routed row r: gather[r] / topk (NULL: r)
    int topk;
    int src_rows;
    const int32_t* offsets;   // [E + 1]
    int E;
    int rows;
    const uint8_t* W;         // expert 0: blob (GF_I8) or rows [N, K] (16 bit)
    size_t expert_stride;     // bytes between experts
    unsigned ldw;             // 16 bit: bytes between rows of W
    size_t codes_off, scales_off;   // GF_I8: blob sections
    int kb;                   // bytes of K in a row
    int N;                    // columns of Y (paired form: of h; W then holds 2 N rows, gate rows first)
    void* Y;
    size_t ldy;               // elements
    int out;                  // w4a8_dtype of Y
    int lo, hi;               // this launch serves the experts with lo <= rows < hi
};

typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

template <int FMT>
struct GroupedAcc {
    using type = v4f;
};
template <>
struct GroupedAcc<GF_I8> {
    using type = v4i;
};

// One 64-byte MFMA step of a 16 x 16 tile.  w holds 16 bytes of weight column lane % 16, x 16 bytes of token row
// lane % 16; lane / 16 selects which 16 of the step's 64 bytes, the same ones in both.  The weights are the first
// operand, so a lane's four sums are the columns 4 (lane / 16) .. + 3 of token row lane % 16: neighbours in Y.
template <int FMT>
__device__ __forceinline__ typename GroupedAcc<FMT>::type grouped_mfma(const v4i w, const v4i x,
                                                                      const typename GroupedAcc<FMT>::type c) {
    if constexpr (FMT == GF_I8) return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, c, 0, 0, 0);
    else if constexpr (FMT == GF_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w), __builtin_bit_cast(v8bf, x), c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, w), __builtin_bit_cast(v8h, x), c, 0, 0, 0);
}

// Round to nearest even; float16 results past 65504 become infinities, as the conversion does.
__device__ __forceinline__ uint32_t f32_to_f16_rne(float f) {
    return uint32_t(__builtin_bit_cast(uint16_t, static_cast<_Float16>(f)));
}

// silu(g) = g / (1 + exp(-g)), from e = exp(-|g|) <= 1: g / (1 + e), or g e / (1 + e) for g < 0, so that nothing
// overflows and the denominator is in [1, 2].  The exponent's product is formed in two parts; with v_exp_f32 and v_rcp_f32
// (one unit each) the result is good to about 4 units of float32, well inside the half step of the 16-bit types it is
// rounded to.  (The library expf and an IEEE division took 6 us of every 125 us tile of the gate/up product.)
__device__ __forceinline__ float silu_gate(float g) {
    const float a = fmaxf(-fabsf(g), -200.0f), t = a * 1.44269502f;    // exp(-200) is 0 in float32
    const float r = fmaf(a, 1.44269502f, -t) + a * 1.92596303e-8f;     // log2(e) = 1.44269502 + 1.926e-8
    float e = __builtin_amdgcn_exp2f(t);
    e = fmaf(e, r * 0.693147182f, e);
    return (g < 0.0f ? g * e : g) * __builtin_amdgcn_rcpf(1.0f + e);
}

// Two values rounded to nearest even and packed (v_cvt_pk_bf16_f32; NaN stays NaN).
__device__ __forceinline__ uint32_t f32_to_bf16_pair(float lo, float hi) {
    typedef float v2f __attribute__((ext_vector_type(2)));
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{lo, hi}, v2bf));
}
__device__ __forceinline__ uint32_t f32_to_f16_pair(float lo, float hi) {
    return f32_to_f16_rne(lo) | (f32_to_f16_rne(hi) << 16);
}

// Four neighbouring outputs of one row, of which n (1..4) exist.  A whole quad goes out in one store wherever it starts:
// global memory takes wide stores at any element's address.
__device__ __forceinline__ void grouped_store(const GroupedArgs& a, const size_t at, const int n, const float y0,
                                              const float y1, const float y2, const float y3) {
    typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
    typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
    if (a.out == W4A8_F32) {
        float* p = static_cast<float*>(a.Y) + at;
        if (n == 4) {
            *reinterpret_cast<f4*>(p) = f4{y0, y1, y2, y3};
        } else {
            p[0] = y0;
            if (n > 1) p[1] = y1;
            if (n > 2) p[2] = y2;
        }
        return;
    }
    const bool f16 = a.out == W4A8_F16;
    const uint32_t lo = f16 ? f32_to_f16_pair(y0, y1) : f32_to_bf16_pair(y0, y1);
    const uint32_t hi = f16 ? f32_to_f16_pair(y2, y3) : f32_to_bf16_pair(y2, y3);
    uint16_t* p = static_cast<uint16_t*>(a.Y) + at;
    if (n == 4) {
        *reinterpret_cast<u2*>(p) = u2{lo, hi};
    } else {
        p[0] = uint16_t(lo);
        if (n > 1) p[1] = uint16_t(lo >> 16);
        if (n > 2) p[2] = uint16_t(hi);
    }
}

// Source row of routed row r, or -1 (a gather entry that names no row of X: its output is zero).
__device__ __forceinline__ int grouped_src(const GroupedArgs& a, int r) {
    if (!a.gather) return r;
    const int g = a.gather[r];
    if (g < 0) return -1;
    const int t = g / a.topk;
    return t < a.src_rows ? t : -1;
}

// MFMA tiles (w4a8_moe_grouped_tile_kernels.hip) over the experts with a.lo <= rows < a.hi; returns whether small ones.
struct TileChoice {
    bool small;
    double us;
};
TileChoice choose_tiles(const GroupedArgs& a, bool i8, bool pair);
bool launch_grouped_tile(const GroupedArgs& a, int fmt, bool pair, hipStream_t s);

}  // namespace w4a8
