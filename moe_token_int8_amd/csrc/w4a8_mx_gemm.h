// Products of MX activations with packed MXFP4 weights: arguments, the scaled MFMA and the outputs, shared by the streaming and
// the tile kernels (gfx950).
#pragma once

#include "w4a8_mx.h"
#include "w4a8_moe_grouped.h"

namespace w4a8 {

struct MxArgs {
    const uint8_t* X;         // activation codes, rows of rowb bytes
    const uint8_t* sx;        // their scale bytes, rows of 4 K1
    unsigned rowb;
    const int32_t* gather;    // source row of routed row r: gather[r] / k (NULL: r)
    unsigned div_mul;         // x / k = (umulhi(x, div_mul) + x) >> div_shift for x < 2^31
    int div_shift;
    int src_rows;
    const int32_t* offsets;   // [E + 1] (NULL: one expert, all rows: the dense product)
    int E;
    int rows;
    const uint8_t* W;         // packed weights of expert 0
    size_t expert_stride;     // bytes between experts
    size_t scales_off;
    int K1;                   // steps of 128 k
    int N;                    // columns of Y (paired form: of h; W then has 2 N, gate columns first)
    void* Y;
    size_t ldy;               // elements
    int out;                  // w4a8_dtype of Y
    uint8_t* Hq;              // paired form: codes and scales of h in place of Y (h_fmt; NULL: Y)
    uint8_t* sh;
    int h_fmt;
};

typedef int v8i __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int mx_row_first(const MxArgs& a, int e) {
    return a.offsets ? min(max(a.offsets[e], 0), a.rows) : 0;
}
__device__ __forceinline__ int mx_row_last(const MxArgs& a, int e) {
    return a.offsets ? min(max(a.offsets[e + 1], 0), a.rows) : a.rows;
}

// Scales of the two gate and the two up tiles of a wave in the paired form, where the first gate tile is even.  The gate tiles' bytes
// are in one word, the up tiles' in one or two (in the second, b, only if the first up tile is the last of its four).
struct MxPairScales {
    unsigned gate, up, up2;   // byte offsets of the words in the scales of step 0; NONE: not needed
    int gshift, ubyte;        // where the two bytes are
};
template <unsigned NONE>
__device__ __forceinline__ MxPairScales mx_pair_scales(const MxArgs& a, const int tile, const bool there, const int lane) {
    const int up = tile + a.N / 16;
    const unsigned quad = unsigned(a.K1) * 256u, l = unsigned(lane) * 4u;
    return {there ? unsigned(tile >> 2) * quad + l : NONE, there ? unsigned(up >> 2) * quad + l : NONE,
            there && (up & 3) == 3 && tile + 1 < a.N / 16 ? unsigned((up >> 2) + 1) * quad + l : NONE, (tile & 2) * 8, up & 3};
}

// Inclusive sum over the lanes up to this one: shifts within rows of 16 by DPP, then the rows' last lanes passed on.
__device__ __forceinline__ int wave_prefix(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
    return x;
}

// Token of a gather entry, or -1 if it names no row of X.
__device__ __forceinline__ int mx_token(const MxArgs& a, int g) {
    const int t = int((__umulhi(unsigned(g), a.div_mul) + unsigned(g)) >> a.div_shift);
    return g >= 0 && t < a.src_rows ? t : -1;
}

// Source row of routed row r, or -1 (a gather entry that names no row of X: its output is zero).
__device__ __forceinline__ int mx_src(const MxArgs& a, int r) {
    if (!a.gather) return r;
    return mx_token(a, a.gather[r]);
}

// Operand of one step of 128 k: 16 bytes of fp4 (a lane's block of 32), or two pieces of 16 fp8 values (k = 16 q and k = 64 + 16 q
// of the step, where q = lane / 16).
template <int FMT>
struct MxOperand {
    v4i p[FMT == W4A8_MX_FP4 ? 1 : 2];
};

// Within 8 neighbouring k the MFMA aligns the products of fp8 to the largest one and drops what lies 14 bits and more below its
// operands' exponents (measured: 2688 + 2^-3 is exact, 2^-4 is lost; 8 places further along K it is not), 5e-6 of a sum of normal
// values and 2e-5 with outliers: less than a 16-bit output rounds, but not a sum in 32 bits, and seen where an element of h lies near
// a tie of its code (a layer's error against float64 2.0e-3 in place of 1.7e-3).  So an operand is multiplied in two parts, its elements
// of 2 and more and the smaller ones: the products of a part span no more than 14 bits, and nothing is dropped.

// The elements of magnitude 2 and more (bit 6 of their byte, the high bit of the exponent, is set); the others are zero.
__device__ __forceinline__ v4i mx_large(const v4i x) {
    v4i r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // v_perm_b32 makes 255 of a selector past 12 and takes byte 0 of its operand, which is 0, for 0
        r[i] = x[i] & int(__builtin_amdgcn_perm(0u, 0u, uint32_t(x[i]) & 0x40404040u));
    }
    return r;
}

// One step of a 16 x 16 tile: v_mfma_scale_f32_16x16x128_f8f6f4 multiplies blocks of 32 k with their scales and sums in float32
// (exact where float32 holds the sum, else within 2^-23 of the sum of magnitudes).  The weights are the first operand, so
// a lane's four sums are the columns 4 (lane / 16) .. + 3 of activation row lane % 16.  A lane's scale is that of block lane / 16:
// byte WB of sw, byte 0 of sx.
template <int FMT, int WB>
__device__ __forceinline__ v4f mx_mfma(const v4i w, const MxOperand<FMT>& x, v4f c, const uint32_t sw, const uint32_t sx) {
    const v8i a = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
    if constexpr (FMT == W4A8_MX_FP4) {
        const v8i b = __builtin_shufflevector(x.p[0], x.p[0], 0, 1, 2, 3, -1, -1, -1, -1);
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, WB, int(sw), 0, int(sx));
    } else {
        const v4i l0 = mx_large(x.p[0]), l1 = mx_large(x.p[1]), s0 = x.p[0] ^ l0, s1 = x.p[1] ^ l1;
        const v8i l = __builtin_shufflevector(l0, l1, 0, 1, 2, 3, 4, 5, 6, 7);
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, l, c, 4, 0, WB, int(sw), 0, int(sx));
        const v8i b = __builtin_shufflevector(s0, s1, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 0, WB, int(sw), 0, int(sx));
    }
}

// silu(g) = g / (1 + exp(-g)) with v_exp_f32 and v_rcp_f32: the exponent's product is rounded once, which costs |g| 2^-24 of the
// result (5e-6 at g = -80), well inside the half step of the 16-bit and the quantized outputs it goes to.  Where exp(g) is below
// 2^-126 (g < -87.3) the reciprocal is 0, and the result -0, also of g = -Inf.
__device__ __forceinline__ float mx_silu(float g) {
    const float r = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269502f));
    return r == 0.0f ? -0.0f : g * r;
}

// Four neighbouring outputs of one row, of which n (1..4) exist.
__device__ __forceinline__ void mx_store(const MxArgs& a, const size_t at, const int n, const v4f y) {
    GroupedArgs g;
    g.Y = a.Y;
    g.out = a.out;
    grouped_store(g, at, n, y[0], y[1], y[2], y[3]);
}

// Blocks of h behind column N, up to whole steps of the product that reads h: zeros, written with the last block.
__device__ __forceinline__ void mx_pad_blocks(const MxArgs& a, const int row, const int first, const int tid8) {
    const int Ip = mx_kp(a.N), bytes = a.h_fmt == W4A8_MX_FP4 ? 16 : 32;
    for (int b = first; b < Ip / 32; ++b) {
        if (tid8 * 4 < bytes) *reinterpret_cast<uint32_t*>(a.Hq + (size_t(row) * size_t(Ip / 32) + size_t(b)) * bytes + tid8 * 4) = 0u;
        if (tid8 == 0) a.sh[size_t(row) * size_t(Ip / 32) + b] = 0;
    }
}

// Four neighbouring values y of one block of h, whose other values are with the 8 lanes around (lane ^ 1, ^ 2, ^ 4): codes and
// scale.  All 8 lanes take part.
__device__ __forceinline__ void mx_store_block(const MxArgs& a, const int row, const int block, const int j, const v4f y, const bool store) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(y[i]) & 0x7fffffffu);
    m = mx_quad_max(m);
    m = max(m, uint32_t(__shfl_xor(int(m), 4, 64)));
    const bool fp4 = a.h_fmt == W4A8_MX_FP4;
    const uint32_t byte = fp4 ? mx_scale_byte<W4A8_MX_FP4>(m) : mx_scale_byte<W4A8_MX_FP8>(m);
    const float up = byte == 255u ? 0.0f : mx_up(byte);
    const v4f v = y * up;
    if (!store) return;
    const size_t at = size_t(row) * size_t(mx_kp(a.N) / 32) + size_t(block);
    if (fp4) {
        const uint32_t q = byte == 255u ? 0u : mx_fp4x4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<uint16_t*>(a.Hq + at * 16 + j * 2) = uint16_t(q);
    } else {
        const uint32_t q = byte == 255u ? 0u : mx_fp8x4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<uint32_t*>(a.Hq + at * 32 + j * 4) = q;
    }
    if (j == 0) a.sh[at] = uint8_t(byte);
}

// MFMA tiles (w4a8_mx_tile_kernels.hip): 128 x 512, 128 x 256, 64 x 256, 32 x 256 or 32 x 128.
enum MxTile { MX_TILE_WIDE, MX_TILE_128, MX_TILE_64, MX_TILE_32, MX_TILE_SMALL };
void launch_mx_tile(const MxArgs& a, int fmt, bool pair, MxTile v, hipStream_t s);

// Routing (the results of w4a8_moe_align) and the codes of the M bfloat16 rows of X in one launch (w4a8_mx_quant_kernels.hip).
void launch_route_quant(const int32_t* ids, int R, int E, int32_t* rows, int32_t* offs, int32_t* inv, const void* X, int M, int K,
                        int fmt, uint8_t* Xq, uint8_t* sx, hipStream_t s);

}  // namespace w4a8
