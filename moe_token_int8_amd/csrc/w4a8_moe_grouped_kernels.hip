// Expert-grouped GEMMs whose experts are 8-bit per-channel blobs (W8A8) or unquantized 16-bit matrices (W16A16): the
// streaming kernel, the launches and the C entry points.
//
// Sources (cited with the page's own section names):
//   P1 "Kimi 2.7 MoE: from 4-bit storage to INT8 (W4A8)" (pwwt.cn), section 4.4: the grouped expert GEMM; section 5.3:
//      W8A8 and 16-bit beside W4A8; section 8: sensitive experts kept in a finer format.
//   P5 "Inference quantization, chapter 1: the Linear layer" (sgdbs.github.io), section 8.3: the per-token x per-channel
//      epilogue Y[i, j] = s_x[i] s_w[j] acc[i, j].
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstring>

#include "w4a8_internal.h"
#include "w4a8_moe_grouped.h"

namespace w4a8 {

// Streaming kernel: experts with few rows, bound by the read of their weights.
//
// A workgroup of 8 waves owns one tile of up to 16 * MS routed rows of one expert and 64 weight columns (4 MFMA tiles; the
// paired form: 32 gate columns and the matching 32 up columns) over all of K.  The waves share K: wave w takes the
// 128-byte units w, w + 8, w + 16, ... of every row, so that at any time the workgroup reads 1 KiB runs of each weight
// row (16 KiB runs of a packed tile), and no operand is used by two waves: weights and activations go from memory to
// registers in the layout of the MFMA operands, with no LDS and no barrier in the loop.  D units of 8 + 2 MS loads are in
// flight per wave.  At the end the 8 partial sums are added in wave order through LDS (int32 sums exactly).
constexpr int GS_WAVES = 8;
constexpr int GS_CT = 4;                                        // column tiles of a workgroup

// Byte within a 128-byte unit of the 16 bytes that lane group q holds in half h.  Packed codes: the layout's
// k = 64 h + 16 q.  Row-major: 32 q + 16 h, so that a lane reads 32 neighbouring bytes; the order of k within a unit is
// free as long as both operands have the same.
template <int FMT>
__device__ __forceinline__ unsigned unit_byte(int q, int h) {
    return FMT == GF_I8 ? unsigned(64 * h + 16 * q) : unsigned(32 * q + 16 * h);
}

template <int FMT, bool PAIR, int MS, int D>
__global__ __launch_bounds__(512, MS == 1 ? 4 : 2) void moe_grouped_stream_kernel(GroupedArgs a, int ncb) {
    using acc_t = typename GroupedAcc<FMT>::type;
    constexpr int CT = GS_CT, COLS = PAIR ? 32 : 64;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = int(blockIdx.x) / ncb, cb = int(blockIdx.x) - slot * ncb;
    TileRows tr;
    {
        GemmArgs g;                                             // moe_tile reads these members only
        g.offsets = a.offsets;
        g.E = a.E;
        g.M = a.rows;
        g.moe_lo = a.lo;
        g.moe_hi = a.hi;
        tr = moe_tile<16 * MS>(g, slot, lane);
    }
    const int expert = __builtin_amdgcn_readfirstlane(tr.expert);
    if (expert < 0) return;                                     // uniform over the workgroup
    const int rbeg = __builtin_amdgcn_readfirstlane(tr.rbeg), nrows = __builtin_amdgcn_readfirstlane(tr.rend) - rbeg;
    const int q = lane >> 4, c16 = lane & 15;
    const int units = (a.kb + 127) / 128;

    // activation rows of this lane; rows past the tile repeat its first row (their sums are not stored)
    const uint8_t* xrow[MS];
#pragma unroll
    for (int ms = 0; ms < MS; ++ms) {
        const int row = ms * 16 + c16;
        const int src = grouped_src(a, rbeg + (row < nrows ? row : 0));
        xrow[ms] = a.X + size_t(src < 0 ? 0 : src) * size_t(a.ldx);
    }

    // weights: one buffer descriptor that ends with the last byte this workgroup may read (paired form: one for the
    // gate and one for the up rows); offsets past it load zeros
    const uint8_t* wexp = a.W + size_t(expert) * a.expert_stride;
    __amdgpu_buffer_rsrc_t wr[PAIR ? 2 : 1];
    unsigned woff[CT];                                          // of this lane in each tile
    constexpr unsigned NONE = 0x7ffffff0u;
    if constexpr (FMT == GF_I8) {
        const int tile0 = cb * CT, ntiles = (a.N + 15) / 16;
        const unsigned tile_bytes = unsigned(units) * 2048u;
        wr[0] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(wexp + a.codes_off + size_t(tile0) * tile_bytes), 0,
                                                  int(unsigned(min(CT, ntiles - tile0)) * tile_bytes), 0x00020000);
#pragma unroll
        for (int t = 0; t < CT; ++t) woff[t] = tile0 + t < ntiles ? t * tile_bytes + lane * 32u : NONE;
    } else {
        const int n0 = cb * COLS, nvalid = min(COLS, a.N - n0);
        const unsigned extent = unsigned(nvalid - 1) * a.ldw + unsigned(a.kb);
#pragma unroll
        for (int p = 0; p < (PAIR ? 2 : 1); ++p)
            wr[p] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(wexp + (size_t(n0) + (p ? a.N : 0)) * a.ldw), 0,
                                                      int(extent), 0x00020000);
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            const int col = (PAIR ? t & 1 : t) * 16 + c16;
            woff[t] = col < nvalid ? unsigned(col) * a.ldw : NONE;
        }
    }

    v4i wv[D][CT][2], xv[D][MS][2];
    auto load = [&](const int d, const int u) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const unsigned b = unsigned(u) * 128u + unit_byte<FMT>(q, h);
            const bool in = b < unsigned(a.kb);
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                unsigned off;
                if constexpr (FMT == GF_I8) off = in && woff[t] != NONE ? woff[t] + unsigned(u) * 2048u + 16u * h : NONE;
                else off = in && woff[t] != NONE ? woff[t] + b : NONE;
                wv[d][t][h] = __builtin_amdgcn_raw_buffer_load_b128(wr[PAIR ? t >> 1 : 0], off, 0, 2);
            }
#pragma unroll
            for (int ms = 0; ms < MS; ++ms) xv[d][ms][h] = *reinterpret_cast<const v4i*>(xrow[ms] + (in ? b : 0u));
        }
    };
    acc_t acc[CT][MS];
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int ms = 0; ms < MS; ++ms) acc[t][ms] = acc_t{};

#pragma unroll
    for (int d = 0; d < D; ++d) load(d, wave + d * GS_WAVES);
    for (int u = wave; u < units; u += D * GS_WAVES) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int ud = u + d * GS_WAVES;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // 16-bit values past the end of K: the weights are zero, and the activations have to be, since
                // the bytes loaded in their place may hold an infinity or a NaN
                const bool in = FMT == GF_I8 || unsigned(ud) * 128u + unit_byte<FMT>(q, h) < unsigned(a.kb);
#pragma unroll
                for (int ms = 0; ms < MS; ++ms) {
                    v4i x = xv[d][ms][h];
                    if constexpr (FMT != GF_I8) x = in ? x : v4i{0, 0, 0, 0};
#pragma unroll
                    for (int t = 0; t < CT; ++t) acc[t][ms] = grouped_mfma<FMT>(wv[d][t][h], x, acc[t][ms]);
                }
            }
            load(d, ud + D * GS_WAVES);
        }
    }

    // the 8 partial sums: planes of 16 bytes a lane, [wave][tile][row block][lane]
    acc_t* red = reinterpret_cast<acc_t*>(smem);
    constexpr int ITEMS = CT * MS * 64;
    constexpr int KEPT = MS == 4 ? 4 : GS_WAVES;                // planes held at a time
    if constexpr (KEPT < GS_WAVES) {
        if (wave >= KEPT) {
#pragma unroll
            for (int t = 0; t < CT; ++t)
#pragma unroll
                for (int ms = 0; ms < MS; ++ms) red[(wave - KEPT) * ITEMS + (t * MS + ms) * 64 + lane] = acc[t][ms];
        }
        lds_barrier();
        if (wave < KEPT) {
#pragma unroll
            for (int t = 0; t < CT; ++t)
#pragma unroll
                for (int ms = 0; ms < MS; ++ms) acc[t][ms] += red[wave * ITEMS + (t * MS + ms) * 64 + lane];
        }
    }
    if (wave < KEPT) {                                          // own plane: nobody else reads it before the barrier
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int ms = 0; ms < MS; ++ms) red[wave * ITEMS + (t * MS + ms) * 64 + lane] = acc[t][ms];
    }
    lds_barrier();
    auto total = [&](const int item) __attribute__((always_inline)) {
        acc_t s = red[item];
#pragma unroll
        for (int w = 1; w < KEPT; ++w) s += red[w * ITEMS + item];
        return s;
    };
    const bool wide = grouped_wide(a);
    for (int item = tid; item < (PAIR ? ITEMS / 2 : ITEMS); item += 512) {
        const int l = item & 63, ms = (item >> 6) % MS, t = (item >> 6) / MS;
        const int row = ms * 16 + (l & 15), col = cb * COLS + t * 16 + 4 * (l >> 4);
        if (row >= nrows || col >= a.N) continue;
        const acc_t s = total(item);
        const int src = grouped_src(a, rbeg + row);
        float y[4];
        if constexpr (FMT == GF_I8) {
            const float sxr = src < 0 ? 0.0f : a.sx[src];
            const float4 sw = *reinterpret_cast<const float4*>(wexp + a.scales_off + size_t(col) * 4);
            y[0] = (float(s[0]) * sw.x) * sxr;
            y[1] = (float(s[1]) * sw.y) * sxr;
            y[2] = (float(s[2]) * sw.z) * sxr;
            y[3] = (float(s[3]) * sw.w) * sxr;
        } else if constexpr (PAIR) {
            const acc_t up = total(item + ITEMS / 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = src < 0 ? 0.0f : silu_gate(s[i]) * up[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = src < 0 ? 0.0f : s[i];
        }
        grouped_store(a, size_t(rbeg + row) * a.ldy + col, min(4, a.N - col), wide, y[0], y[1], y[2], y[3]);
    }
}

template <int FMT, bool PAIR, int MS, int D>
static void launch_stream_t(const GroupedArgs& a, long long slots, hipStream_t s) {
    constexpr size_t lds = size_t(MS == 4 ? 4 : GS_WAVES) * GS_CT * MS * 64 * 16;
    static_assert(lds <= 65536, "two workgroups of 16-row tiles share a compute unit");
    const int ncb = (a.N + (PAIR ? 31 : 63)) / (PAIR ? 32 : 64);
    moe_grouped_stream_kernel<FMT, PAIR, MS, D><<<dim3(unsigned(slots * ncb)), dim3(512), lds, s>>>(a, ncb);
}

// Row classes of the streaming kernel, one launch each: an expert of up to 16 rows costs nothing for rows it does not
// have, and the launches of classes that no expert can be in are left out.  `slots` bounds the row tiles of the class.
template <int FMT, bool PAIR>
static void launch_grouped(GroupedArgs a, hipStream_t s) {
    const long long rows = a.rows, E = a.E;
    a.lo = 1, a.hi = 17;
    launch_stream_t<FMT, PAIR, 1, 2>(a, std::min(E, rows), s);
    if (rows > 16) {
        a.lo = 17, a.hi = 33;
        launch_stream_t<FMT, PAIR, 2, 2>(a, std::min(E, rows / 17), s);
    }
    // the MFMA-tile kernel reaches activation rows through 32-bit offsets from X (gathered) or from its tile's first row
    const bool near = a.ldx <= (1 << 24) && (!a.gather || (long long)a.src_rows * a.ldx < (1ll << 32) - 256);
    if (rows > 32) {
        a.lo = 33, a.hi = near ? 65 : 0x7fffffff;
        launch_stream_t<FMT, PAIR, 4, 2>(a, near ? std::min(E, rows / 33) : rows / 64 + std::min(E, rows / 33), s);
    }
    if (rows > 64 && near) {
        a.lo = 65, a.hi = 0x7fffffff;
        launch_grouped_tile(a, FMT, PAIR, s);
    }
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static int launched() { return hipGetLastError() == hipSuccess ? W4A8_OK : W4A8_EHIP; }

// Columns a launch may have: blocks = slots * column blocks stay below 2^31 for 2^24 rows.
constexpr int GROUPED_MAX_N = 1 << 20;
constexpr int GROUPED_MAX_ROWS = 1 << 24;

// Blob of 8-bit codes with one float32 scale per channel.
static int check_w8(const w4a8_wdesc* d) {
    const int st = desc_status(d);
    if (st) return st;
    const Layout L = layout_of(d);
    if (L.bits != 8 || L.G != 1 || L.sbytes != 4) return W4A8_EUNSUPPORTED;
    // one int32 accumulator over all of K, and 32-bit offsets within a blob's codes
    if (int64_t(L.K) * 127 * 127 >= (int64_t(1) << 31) || L.codes_bytes >= (size_t(1) << 31) || L.N > GROUPED_MAX_N)
        return W4A8_EUNSUPPORTED;
    return W4A8_OK;
}

static int check_w8_call(const int8_t* Xq, const float* sx, const int32_t* gather, int k, const int32_t* offsets, int E,
                         int rows, int src_rows, const void* blobs, size_t stride, const w4a8_wdesc* d, const void* Y,
                         int out_dtype) {
    const int st = check_w8(d);
    if (st) return st;
    if (rows < 0 || src_rows < 0 || E <= 0 || E > 1024 || (out_dtype != W4A8_BF16 && out_dtype != W4A8_F32)) return W4A8_EINVAL;
    if (rows == 0) return W4A8_OK;
    if (rows > GROUPED_MAX_ROWS) return W4A8_EUNSUPPORTED;
    if (!Xq || !sx || !offsets || !blobs || !Y) return W4A8_EINVAL;
    if (gather ? (k <= 0 || src_rows == 0) : src_rows < rows) return W4A8_EINVAL;
    if (E > 1 && stride < layout_of(d).total) return W4A8_EINVAL;
    if (!aligned16(Xq) || !aligned16(blobs) || (stride & 15)) return W4A8_EINVAL;
    if (reinterpret_cast<uintptr_t>(Y) & (out_dtype == W4A8_F32 ? 3u : 1u)) return W4A8_EINVAL;
    return W4A8_OK;
}

static int check_w16_call(const void* X, int dtype, int ldx, const int32_t* gather, int k, const int32_t* offsets, int E,
                          int rows, int src_rows, const void* W, size_t stride, int ldw, int K, int N, bool pair,
                          const void* Y, int ldy, int out_dtype) {
    if (dtype != W4A8_BF16 && dtype != W4A8_F16) return W4A8_EINVAL;
    if (out_dtype != dtype && (pair || out_dtype != W4A8_F32)) return W4A8_EINVAL;
    if (rows < 0 || src_rows < 0 || E <= 0 || E > 1024 || K <= 0 || N <= 0) return W4A8_EINVAL;
    if (K % 8 || ldx % 8 || ldw % 8 || stride % 8 || ldx < K || ldw < K || ldy < N) return W4A8_EINVAL;
    if (E > 1 && stride < (size_t(N) * (pair ? 2 : 1) - 1) * size_t(ldw) + size_t(K)) return W4A8_EINVAL;
    if (N > GROUPED_MAX_N || ldw > (1 << 23) || rows > GROUPED_MAX_ROWS) return W4A8_EUNSUPPORTED;
    if (rows == 0) return W4A8_OK;
    if (!X || !offsets || !W || !Y) return W4A8_EINVAL;
    if (gather ? (k <= 0 || src_rows == 0) : src_rows < rows) return W4A8_EINVAL;
    if (!aligned16(X) || !aligned16(W) || (reinterpret_cast<uintptr_t>(Y) & (out_dtype == W4A8_F32 ? 3u : 1u)))
        return W4A8_EINVAL;
    return W4A8_OK;
}

static int run_w8(const int8_t* Xq, const float* sx, const int32_t* gather, int k, const int32_t* offsets, int E, int rows,
                  int src_rows, const void* blobs, size_t stride, const w4a8_wdesc* d, void* Y, int out_dtype,
                  hipStream_t s) {
    const Layout L = layout_of(d);
    if (log_on())
        std::fprintf(stderr, "w4a8: w4a8_moe_gemm_w8a8 E=%d rows=%d K=%d N=%d -> moe_grouped_stream_kernel\n", E, rows, L.K,
                     L.N);
    GroupedArgs a;
    std::memset(&a, 0, sizeof(a));
    a.X = reinterpret_cast<const uint8_t*>(Xq);
    a.ldx = L.K;
    a.sx = sx;
    a.gather = gather;
    a.topk = k;
    a.src_rows = src_rows;
    a.offsets = offsets;
    a.E = E;
    a.rows = rows;
    a.W = static_cast<const uint8_t*>(blobs);
    a.expert_stride = stride;
    a.codes_off = L.codes_off;
    a.scales_off = L.scales_off;
    a.kb = L.K;
    a.N = L.N;
    a.Y = Y;
    a.ldy = size_t(L.N);
    a.out = out_dtype;
    launch_grouped<GF_I8, false>(a, s);
    return launched();
}

static int run_w16(const void* X, int dtype, int ldx, const int32_t* gather, int k, const int32_t* offsets, int E, int rows,
                   int src_rows, const void* W, size_t stride, int ldw, int K, int N, bool pair, void* Y, int ldy,
                   int out_dtype, hipStream_t s) {
    if (log_on())
        std::fprintf(stderr, "w4a8: w4a8_moe_gemm%s_w16a16 E=%d rows=%d K=%d N=%d %s -> moe_grouped_stream_kernel\n",
                     pair ? "_silu" : "", E, rows, K, N, dtype == W4A8_F16 ? "float16" : "bfloat16");
    GroupedArgs a;
    std::memset(&a, 0, sizeof(a));
    a.X = static_cast<const uint8_t*>(X);
    a.ldx = 2ll * ldx;
    a.gather = gather;
    a.topk = k;
    a.src_rows = src_rows;
    a.offsets = offsets;
    a.E = E;
    a.rows = rows;
    a.W = static_cast<const uint8_t*>(W);
    a.expert_stride = 2 * stride;
    a.ldw = 2u * unsigned(ldw);
    a.kb = 2 * K;
    a.N = N;
    a.Y = Y;
    a.ldy = size_t(ldy);
    a.out = out_dtype;
    if (dtype == W4A8_BF16) {
        if (pair) launch_grouped<GF_BF16, true>(a, s);
        else launch_grouped<GF_BF16, false>(a, s);
    } else {
        if (pair) launch_grouped<GF_F16, true>(a, s);
        else launch_grouped<GF_F16, false>(a, s);
    }
    return launched();
}

}  // namespace w4a8

using namespace w4a8;

extern "C" {

int w4a8_moe_gemm_w8a8(const int8_t* Xq, const float* sx, const int32_t* gather, int k, const int32_t* offsets, int E,
                       int rows, int src_rows, const void* blobs, size_t stride, const w4a8_wdesc* d, void* Y, int out_dtype,
                       void* stream) {
    const int st = check_w8_call(Xq, sx, gather, k, offsets, E, rows, src_rows, blobs, stride, d, Y, out_dtype);
    if (st || rows == 0) return st;
    return run_w8(Xq, sx, gather, k, offsets, E, rows, src_rows, blobs, stride, d, Y, out_dtype,
                  static_cast<hipStream_t>(stream));
}

int w4a8_moe_gemm_w16a16(const void* X, int dtype, int ldx, const int32_t* gather, int k, const int32_t* offsets, int E,
                         int rows, int src_rows, const void* W, size_t stride, int ldw, int K, int N, void* Y, int ldy,
                         int out_dtype, void* stream) {
    const int st = check_w16_call(X, dtype, ldx, gather, k, offsets, E, rows, src_rows, W, stride, ldw, K, N, false, Y, ldy,
                                  out_dtype);
    if (st || rows == 0) return st;
    return run_w16(X, dtype, ldx, gather, k, offsets, E, rows, src_rows, W, stride, ldw, K, N, false, Y, ldy, out_dtype,
                   static_cast<hipStream_t>(stream));
}

int w4a8_moe_gemm_silu_w16a16(const void* X, int dtype, int ldx, const int32_t* gather, int k, const int32_t* offsets, int E,
                              int rows, int src_rows, const void* W, size_t stride, int ldw, int K, int I, void* H, int ldh,
                              void* stream) {
    const int st = check_w16_call(X, dtype, ldx, gather, k, offsets, E, rows, src_rows, W, stride, ldw, K, I, true, H, ldh,
                                  dtype);
    if (st || rows == 0) return st;
    return run_w16(X, dtype, ldx, gather, k, offsets, E, rows, src_rows, W, stride, ldw, K, I, true, H, ldh, dtype,
                   static_cast<hipStream_t>(stream));
}

}  // extern "C"
