// Products of MX activations (MXFP4 or MXFP8) with packed MXFP4 weights, dense and by expert: the streaming kernel, the launches,
// the C entry points and the expert layer.
//
// Sources (cited with the page's own section names):
//   P1 "Kimi 2.7 MoE: from 4-bit storage to INT8 (W4A8)" (pwwt.cn), section 4.4: the grouped expert GEMM and the steps of the
//      layer; section 5.1: tiles matched to the MFMA operands.
//   P3 "Quantization: formats, error and the real execution path" (wineandchord.com): FP4 / FP8 with block scales.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstring>

#include "w4a8_mx_gemm.h"

namespace w4a8 {

// Streaming kernel: few rows, bound by the read of the weights.
//
// A workgroup of 8 waves owns one tile of up to 16 MS rows of one expert and CT MFMA tiles of 16 weight columns (paired form:
// gate columns in half of them, the matching up columns in the others) over all of K.  The waves share K in units of U steps:
// wave w takes the units w, w + 8, ...; weights and activations go from memory to registers in the layout of the MFMA operands
// (a step of a weight tile is one contiguous KiB), with no LDS and no barrier in the loop, and the loads of a wave's next unit
// are in flight while it multiplies.  The 8 partial sums are added in wave order through LDS, so a call repeats bit for bit.
constexpr int MXS_WAVES = 8;

template <int MT>
__device__ __forceinline__ TileRows mx_find(const MxArgs& a, int slot, int lane) {
    TileRows tr{0, 0, -1};
    if (!a.offsets) {
        if ((long long)slot * MT < a.rows) tr = {slot * MT, min(a.rows, slot * MT + MT), 0};
        return tr;
    }
    int base = 0;
    for (int c0 = 0; c0 < a.E; c0 += 256) {                     // the offsets of 256 experts are requested together
        int b[4], e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int x = c0 + j * 64 + lane;
            b[j] = x < a.E ? a.offsets[x] : 0;
            e[j] = x < a.E ? a.offsets[x + 1] : 0;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // malformed offsets cannot move a tile outside the rows of the call
            const int e0 = min(max(b[j], 0), a.rows), e1 = min(max(e[j], e0), a.rows), cnt = e1 - e0;
            const int t = cnt >= a.lo && cnt < a.hi ? (cnt + MT - 1) / MT : 0;
            int incl = t;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int y = __shfl_up(incl, o, 64);
                if (lane >= o) incl += y;
            }
            const unsigned long long hit = __ballot(slot >= base + incl - t && slot < base + incl);
            if (hit) {
                const int src = __ffsll((long long)hit) - 1;
                tr.expert = c0 + j * 64 + src;
                tr.rbeg = __builtin_amdgcn_readlane(e0 + (slot - base - (incl - t)) * MT, src);
                tr.rend = min(__builtin_amdgcn_readlane(e1, src), tr.rbeg + MT);
                return tr;
            }
            base += __builtin_amdgcn_readlane(incl, 63);
        }
    }
    return tr;
}

template <int FMT, bool PAIR, int MS, int CT, bool NT>
__global__ __launch_bounds__(512, 4) void mx_stream_kernel(MxArgs a, int ncb) {
    constexpr int U = 2;                                        // steps of a unit
    constexpr int COLS = PAIR ? CT * 8 : CT * 16;
    constexpr bool QUADS = !PAIR && CT == 4;                    // the scales of the 4 tiles are one word
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, c16 = lane & 15;
    const int units = (a.K1 + U - 1) / U;
    const unsigned tile_bytes = unsigned(a.K1) * 1024u, quad_bytes = unsigned(a.K1) * 256u;
    for (unsigned item = blockIdx.x;; item += gridDim.x) {
        const int slot = int(item / unsigned(ncb)), cb = int(item - unsigned(slot) * unsigned(ncb));
        const TileRows tr = mx_find<16 * MS>(a, slot, lane);
        const int expert = __builtin_amdgcn_readfirstlane(tr.expert);
        if (expert < 0) return;                                 // uniform over the workgroup; no later slot has a tile
        const int rbeg = __builtin_amdgcn_readfirstlane(tr.rbeg), nrows = __builtin_amdgcn_readfirstlane(tr.rend) - rbeg;

        // weights and their scales: descriptors that end with the expert's; offsets past them load zeros, which is what tiles
        // past the last column and steps past the last of K take
        const uint8_t* wexp = a.W + size_t(expert) * a.expert_stride;
        const int width = PAIR ? 2 * a.N : a.N, ntiles = (width + 15) / 16;
        const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(wexp), 0,
                                                                            int(unsigned(ntiles) * tile_bytes), 0x00020000);
        const __amdgpu_buffer_rsrc_t sr = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(wexp + a.scales_off), 0, int(unsigned((width + 63) / 64) * quad_bytes), 0x00020000);
        constexpr unsigned NONE = 0x80000000u;
        int tile[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t)
            tile[t] = PAIR ? cb * (CT / 2) + t % (CT / 2) + (t >= CT / 2 ? a.N / 16 : 0) : cb * CT + t;
        const uint8_t* xrow[MS];
        const uint8_t* srow[MS];
        struct Unit {
            v4i w[U][CT];
            uint32_t sw[U][QUADS ? 1 : CT];
            MxOperand<FMT> x[U][MS];
            uint32_t sx[U][MS];
        };
        // NT: the non-temporal hint, for calls that read more weights than the Infinity Cache holds.
        auto load_w = [&](Unit& b, const int u) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int step = u * U + i;
                const bool in = step < a.K1;
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    const bool there = in && (PAIR ? cb * (CT / 2) + t % (CT / 2) < a.N / 16 : tile[t] < ntiles);
                    b.w[i][t] = __builtin_amdgcn_raw_buffer_load_b128(
                        wr, there ? unsigned(tile[t]) * tile_bytes + unsigned(step) * 1024u + unsigned(lane) * 16u : NONE, 0, NT ? 2 : 0);
                    if (!QUADS)
                        b.sw[i][QUADS ? 0 : t] = __builtin_amdgcn_raw_buffer_load_b8(
                            sr, there ? unsigned(tile[t] >> 2) * quad_bytes + unsigned(step) * 256u + unsigned(lane) * 4u + unsigned(tile[t] & 3)
                                      : NONE, 0, 0);
                }
                if (QUADS)
                    b.sw[i][0] = __builtin_amdgcn_raw_buffer_load_b32(
                        sr, in ? unsigned(cb) * quad_bytes + unsigned(step) * 256u + unsigned(lane) * 4u : NONE, 0, 0);
            }
        };
        auto load_x = [&](Unit& b, const int u) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const unsigned step = unsigned(min(u * U + i, a.K1 - 1));   // past the last step the weights are zero
#pragma unroll
                for (int ms = 0; ms < MS; ++ms) {
                    if constexpr (FMT == W4A8_MX_FP4) {
                        b.x[i][ms].p[0] = *reinterpret_cast<const v4i*>(xrow[ms] + step * 64u + unsigned(q) * 16u);
                    } else {
                        b.x[i][ms].p[0] = *reinterpret_cast<const v4i*>(xrow[ms] + step * 128u + unsigned(q) * 16u);
                        b.x[i][ms].p[1] = *reinterpret_cast<const v4i*>(xrow[ms] + step * 128u + 64u + unsigned(q) * 16u);
                    }
                    b.sx[i][ms] = srow[ms][step * 4u + unsigned(q)];
                }
            }
        };
        // activation rows of this lane; rows past the tile repeat its first row (their sums are not stored)
        int src[MS];
#pragma unroll
        for (int ms = 0; ms < MS; ++ms) {
            const int row = ms * 16 + c16;
            src[ms] = mx_src(a, rbeg + (row < nrows ? row : 0));
        }
        Unit cur, next;
        if (wave < units) load_w(cur, wave);
#pragma unroll
        for (int ms = 0; ms < MS; ++ms) {
            const size_t r = size_t(src[ms] < 0 ? 0 : src[ms]);
            xrow[ms] = a.X + r * a.rowb;
            srow[ms] = a.sx + r * size_t(a.K1) * 4;
        }
        if (wave < units) load_x(cur, wave);

        v4f acc[CT][MS];
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int ms = 0; ms < MS; ++ms) acc[t][ms] = v4f{};
        for (int u = wave; u < units; u += MXS_WAVES) {
            const bool more = u + MXS_WAVES < units;
            if (more) {
                load_w(next, u + MXS_WAVES);
                load_x(next, u + MXS_WAVES);
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int ms = 0; ms < MS; ++ms) {
                    if constexpr (QUADS) {
                        acc[0][ms] = mx_mfma<FMT, 0>(cur.w[i][0], cur.x[i][ms], acc[0][ms], cur.sw[i][0], cur.sx[i][ms]);
                        acc[1][ms] = mx_mfma<FMT, 1>(cur.w[i][1], cur.x[i][ms], acc[1][ms], cur.sw[i][0], cur.sx[i][ms]);
                        acc[2][ms] = mx_mfma<FMT, 2>(cur.w[i][2], cur.x[i][ms], acc[2][ms], cur.sw[i][0], cur.sx[i][ms]);
                        acc[3][ms] = mx_mfma<FMT, 3>(cur.w[i][3], cur.x[i][ms], acc[3][ms], cur.sw[i][0], cur.sx[i][ms]);
                    } else {
#pragma unroll
                        for (int t = 0; t < CT; ++t)
                            acc[t][ms] = mx_mfma<FMT, 0>(cur.w[i][t], cur.x[i][ms], acc[t][ms], cur.sw[i][t], cur.sx[i][ms]);
                    }
                }
            if (more) cur = next;
        }

        // the 8 partial sums: planes of 16 bytes a lane, [wave][tile][row block][lane]
        v4f* red = reinterpret_cast<v4f*>(smem);
        constexpr int ITEMS = CT * MS * 64, OUT = PAIR ? ITEMS / 2 : ITEMS;
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int ms = 0; ms < MS; ++ms) red[wave * ITEMS + (t * MS + ms) * 64 + lane] = acc[t][ms];
        lds_barrier();
        auto total = [&](const int o) __attribute__((always_inline)) {
            v4f s = red[o];
#pragma unroll
            for (int w = 1; w < MXS_WAVES; ++w) s += red[w * ITEMS + o];
            return s;
        };
        constexpr int PER = (OUT + 511) / 512;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int o = tid + i * 512;
            if constexpr (PAIR && CT >= 4) {
                if (a.Hq) {                                     // 8 neighbouring lanes take a row's block of 32 columns
                    constexpr int BL = CT / 4;                  // blocks of a row
                    const int j = o & 7, b = (o >> 3) % BL, row = (o >> 3) / BL, t = b * 2 + (j >> 2);
                    const int at = (t * MS + row / 16) * 64 + (j & 3) * 16 + (row & 15);
                    const int col = cb * COLS + b * 32 + j * 4;
                    const bool in = o < OUT && row < nrows && col < a.N;
                    v4f h{};
                    if (in && mx_src(a, rbeg + row) >= 0) {
                        const v4f g = total(at), u = total(at + ITEMS / 2);
#pragma unroll
                        for (int k = 0; k < 4; ++k) h[k] = silu_gate(g[k]) * u[k];
                    }
                    const bool there = o < OUT && row < nrows && cb * COLS + b * 32 < a.N;
                    mx_store_block(a, rbeg + row, (cb * COLS) / 32 + b, j, h, there);
                    if (there && cb * COLS + b * 32 + 32 >= a.N) mx_pad_blocks(a, rbeg + row, (cb * COLS) / 32 + b + 1, j);
                    continue;
                }
            }
            const int l = o & 63, row = ((o >> 6) % MS) * 16 + (l & 15);
            const int col = cb * COLS + ((o >> 6) / MS) * 16 + 4 * (l >> 4);
            if (o >= OUT || row >= nrows || col >= a.N) continue;
            v4f y = total(o);
            if constexpr (PAIR) {
                const v4f up = total(o + ITEMS / 2);
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = silu_gate(y[k]) * up[k];
            }
            if (mx_src(a, rbeg + row) < 0) y = v4f{};
            mx_store(a, size_t(rbeg + row) * a.ldy + col, min(4, a.N - col), y);
        }
        lds_barrier();                                          // the planes are written again by the next tile
    }
}

// Workgroups of a launch: all tiles up to a bound, beyond which they go round in a grid that is resident at once (two
// workgroups a compute unit).
constexpr long long MXS_GRID = 512;

template <int FMT, bool PAIR, int MS, int CT, bool NT>
static void launch_stream_t(const MxArgs& a, long long slots, hipStream_t s) {
    constexpr size_t lds = size_t(MXS_WAVES) * CT * MS * 64 * 16;
    static_assert(lds <= 65536, "two workgroups share a compute unit");
    constexpr int cols = PAIR ? CT * 8 : CT * 16;
    const int ncb = (a.N + cols - 1) / cols;
    const long long blocks = MS == 1 ? std::min(slots * ncb, 1ll << 22) : std::min(slots * ncb, MXS_GRID);
    mx_stream_kernel<FMT, PAIR, MS, CT, NT><<<dim3(unsigned(blocks)), dim3(512), lds, s>>>(a, ncb);
}

template <int FMT, bool PAIR>
static const char* launch_mx(MxArgs a, hipStream_t s) {
    const long long rows = a.rows, E = a.E;
    a.lo = 1, a.hi = 0x7fffffff;
    if (rows <= 16) {
        launch_stream_t<FMT, PAIR, 1, 4, false>(a, std::min(E, rows), s);
        return "mx_stream_kernel (16-row tiles)";
    }
    launch_stream_t<FMT, PAIR, 2, 4, false>(a, rows / 32 + std::min(E, rows), s);
    return "mx_stream_kernel (32-row tiles)";
}

// out[t] = sum_j w[t, j] Yd[inv[t, j]] in float32, j ascending, rounded once: the experts' outputs stay in float32 (rounded to
// bfloat16 in between, a layer's error against float64 is 2.5e-3 normwise in place of 1.7e-3, that of the one rounding).
// 4 columns a thread; the rows of 8 experts are requested together.
__global__ __launch_bounds__(256) void mx_combine_kernel(const float* Yd, unsigned ldy, const int32_t* inv, const float* w, int k, int H,
                                                         int chunks, uint16_t* out) {
    const int t = int(blockIdx.x / unsigned(chunks)), c = (int(blockIdx.x % unsigned(chunks)) * 256 + int(threadIdx.x)) * 4;
    if (c >= H) return;
    v4f s{};
    for (int j0 = 0; j0 < k; j0 += 8) {
        int row[8];
        float f[8];
        v4f y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            row[j] = j0 + j < k ? inv[size_t(t) * k + j0 + j] : -1;
            f[j] = j0 + j < k ? w[size_t(t) * k + j0 + j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = row[j] >= 0 ? *reinterpret_cast<const v4f*>(Yd + size_t(row[j]) * ldy + c) : v4f{};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (row[j] >= 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = fmaf(f[j], y[j][i], s[i]);
            }
    }
    typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
    uint16_t* p = out + size_t(t) * size_t(H) + c;
    if (c + 4 <= H) {
        *reinterpret_cast<u2*>(p) = u2{f32_to_bf16_pair(s[0], s[1]), f32_to_bf16_pair(s[2], s[3])};
    } else {
        for (int i = 0; i < H - c; ++i) p[i] = uint16_t(f32_to_bf16_rne(s[i]));
    }
}

static bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
static int launched() { return hipGetLastError() == hipSuccess ? W4A8_OK : W4A8_EHIP; }

constexpr int MX_MAX_ROWS = 1 << 24;

// Arguments of every product; width: columns of the weights.
static int check_mx(const void* Xq, const uint8_t* sx, int fmt, const int32_t* gather, int k, const int32_t* offsets, int E, int rows,
                    int src_rows, const void* W, size_t stride, int K, int width) {
    if (fmt != W4A8_MX_FP4 && fmt != W4A8_MX_FP8) return W4A8_EINVAL;
    if (rows < 0 || src_rows < 0 || E <= 0 || E > 1024) return W4A8_EINVAL;
    const int st = mx_check_weights(width, K);
    if (st) return st;
    if (rows > MX_MAX_ROWS || src_rows > MX_MAX_ROWS) return W4A8_EUNSUPPORTED;
    if (rows == 0) return W4A8_OK;
    if (!Xq || !sx || !W || (E > 1 && !offsets)) return W4A8_EINVAL;
    if (gather ? (k <= 0 || src_rows == 0) : src_rows < rows) return W4A8_EINVAL;
    if (E > 1 && stride < mx_layout(width, K).total) return W4A8_EINVAL;
    if (!aligned_to(Xq, 16) || !aligned_to(sx, 4) || !aligned_to(W, 16) || (stride & 15)) return W4A8_EINVAL;
    return W4A8_OK;
}

static int check_out(const void* Y, int ldy, int N, int out, bool f32) {
    if (out != W4A8_BF16 && out != W4A8_F16 && !(f32 && out == W4A8_F32)) return W4A8_EINVAL;
    if (ldy < N || !Y || !aligned_to(Y, out == W4A8_F32 ? 4 : 2)) return W4A8_EINVAL;
    return W4A8_OK;
}

static MxArgs mx_args(const void* Xq, const uint8_t* sx, int fmt, const int32_t* gather, int k, const int32_t* offsets, int E,
                      int rows, int src_rows, const void* W, size_t stride, int K, int width) {
    MxArgs a;
    std::memset(&a, 0, sizeof(a));
    const MxLayout L = mx_layout(width, K);
    a.X = static_cast<const uint8_t*>(Xq);
    a.sx = sx;
    a.rowb = unsigned(mx_row_bytes(fmt, K));
    a.gather = gather;
    a.topk = k;
    a.src_rows = src_rows;
    a.offsets = offsets;
    a.E = E;
    a.rows = rows;
    a.W = static_cast<const uint8_t*>(W);
    a.expert_stride = stride;
    a.scales_off = L.scales_off;
    a.K1 = L.K1;
    return a;
}

// exact: float32 sums of fp8 products that drop nothing.
static int run_mx(const char* call, MxArgs& a, int fmt, bool pair, bool exact, int K, hipStream_t s) {
    const char* names = fmt == W4A8_MX_FP4 ? (pair ? launch_mx<W4A8_MX_FP4, true>(a, s) : launch_mx<W4A8_MX_FP4, false>(a, s))
                        : exact            ? launch_mx<MX_FP8_EXACT, false>(a, s)
                                           : (pair ? launch_mx<W4A8_MX_FP8, true>(a, s) : launch_mx<W4A8_MX_FP8, false>(a, s));
    if (log_on())
        std::fprintf(stderr, "w4a8: %s E=%d rows=%d K=%d N=%d %s -> %s\n", call, a.E, a.rows, K, a.N,
                     fmt == W4A8_MX_FP4 ? "mxfp4" : "mxfp8", names);
    return launched();
}

// Workspace of the layer: pieces in order, each 256-byte aligned.
struct MxLayerWs {
    size_t xq, sx, rows, offs, inv, hq, sh, yd, total;
};
static MxLayerWs mx_layer_ws(int T, int k, int H, int I, int E, int fmt) {
    const size_t R = size_t(T) * size_t(k);
    MxLayerWs w;
    size_t o = 0;
    auto piece = [&](size_t bytes) {
        const size_t at = o;
        o = (o + bytes + 255) & ~size_t(255);
        return at;
    };
    w.xq = piece(size_t(T) * mx_row_bytes(fmt, H)), w.sx = piece(size_t(T) * size_t(mx_kp(H) / 32));
    w.rows = piece(R * 4), w.offs = piece(size_t(E + 1) * 4), w.inv = piece(R * 4);
    w.hq = piece(R * mx_row_bytes(fmt, I)), w.sh = piece(R * size_t(mx_kp(I) / 32));
    w.yd = piece(R * size_t((H + 3) & ~3) * 4);                 // float32, rows at whole 16 bytes
    w.total = o;
    return w;
}

}  // namespace w4a8

using namespace w4a8;

extern "C" {

int w4a8_mx_gemm(const void* Xq, const uint8_t* sx, int fmt, int M, const void* blob, int K, int N, void* Y, int ldy, int out_dtype,
                 void* stream) {
    int st = check_mx(Xq, sx, fmt, nullptr, 1, nullptr, 1, M, M, blob, 0, K, N);
    if (st || M == 0) return st;
    if ((st = check_out(Y, ldy, N, out_dtype, true))) return st;
    MxArgs a = mx_args(Xq, sx, fmt, nullptr, 1, nullptr, 1, M, M, blob, 0, K, N);
    a.N = N, a.Y = Y, a.ldy = size_t(ldy), a.out = out_dtype;
    return run_mx("w4a8_mx_gemm", a, fmt, false, out_dtype == W4A8_F32, K, static_cast<hipStream_t>(stream));
}

int w4a8_moe_gemm_mx(const void* Xq, const uint8_t* sx, int fmt, const int32_t* gather, int k, const int32_t* offsets, int E, int rows,
                     int src_rows, const void* blobs, size_t stride, int K, int N, void* Y, int ldy, int out_dtype, void* stream) {
    int st = check_mx(Xq, sx, fmt, gather, k, offsets, E, rows, src_rows, blobs, stride, K, N);
    if (st || rows == 0) return st;
    if (!offsets) return W4A8_EINVAL;
    if ((st = check_out(Y, ldy, N, out_dtype, true))) return st;
    MxArgs a = mx_args(Xq, sx, fmt, gather, k, offsets, E, rows, src_rows, blobs, stride, K, N);
    a.N = N, a.Y = Y, a.ldy = size_t(ldy), a.out = out_dtype;
    return run_mx("w4a8_moe_gemm_mx", a, fmt, false, out_dtype == W4A8_F32, K, static_cast<hipStream_t>(stream));
}

int w4a8_moe_gemm_silu_mx(const void* Xq, const uint8_t* sx, int fmt, const int32_t* gather, int k, const int32_t* offsets, int E,
                          int rows, int src_rows, const void* blobs, size_t stride, int K, int I, void* H, int ldh, int out_dtype,
                          void* stream) {
    if (I <= 0 || I % 16 || I > MX_MAX_N / 2) return I > MX_MAX_N / 2 ? W4A8_EUNSUPPORTED : W4A8_EINVAL;
    int st = check_mx(Xq, sx, fmt, gather, k, offsets, E, rows, src_rows, blobs, stride, K, 2 * I);
    if (st || rows == 0) return st;
    if (!offsets) return W4A8_EINVAL;
    if ((st = check_out(H, ldh, I, out_dtype, false))) return st;
    MxArgs a = mx_args(Xq, sx, fmt, gather, k, offsets, E, rows, src_rows, blobs, stride, K, 2 * I);
    a.N = I, a.Y = H, a.ldy = size_t(ldh), a.out = out_dtype;
    return run_mx("w4a8_moe_gemm_silu_mx", a, fmt, true, false, K, static_cast<hipStream_t>(stream));
}

int w4a8_moe_gemm_silu_mx_quant(const void* Xq, const uint8_t* sx, int fmt, const int32_t* gather, int k, const int32_t* offsets, int E,
                                int rows, int src_rows, const void* blobs, size_t stride, int K, int I, int h_fmt, void* Hq,
                                uint8_t* sh, void* stream) {
    if (I <= 0 || I % 16 || I > MX_MAX_N / 2) return I > MX_MAX_N / 2 ? W4A8_EUNSUPPORTED : W4A8_EINVAL;
    if (h_fmt != W4A8_MX_FP4 && h_fmt != W4A8_MX_FP8) return W4A8_EINVAL;
    const int st = check_mx(Xq, sx, fmt, gather, k, offsets, E, rows, src_rows, blobs, stride, K, 2 * I);
    if (st || rows == 0) return st;
    if (!offsets || !Hq || !sh || !aligned_to(Hq, 16) || !aligned_to(sh, 4)) return W4A8_EINVAL;
    MxArgs a = mx_args(Xq, sx, fmt, gather, k, offsets, E, rows, src_rows, blobs, stride, K, 2 * I);
    a.N = I, a.Hq = static_cast<uint8_t*>(Hq), a.sh = sh, a.h_fmt = h_fmt;
    return run_mx("w4a8_moe_gemm_silu_mx_quant", a, fmt, true, false, K, static_cast<hipStream_t>(stream));
}

size_t w4a8_moe_mx_workspace_size(int T, int k, int H, int I, int E, int fmt) {
    if (T < 0 || k <= 0 || H <= 0 || I <= 0 || E <= 0 || H > MX_MAX_K || I > MX_MAX_N / 2 ||
        (fmt != W4A8_MX_FP4 && fmt != W4A8_MX_FP8))
        return 0;
    return mx_layer_ws(T, k, H, I, E, fmt).total;
}

int w4a8_moe_forward_mx(const void* X, const int32_t* ids, const float* w, int T, int k, int E, int fmt, const void* gu, size_t gu_stride,
                        const void* dn, size_t d_stride, int H, int I, void* ws, size_t ws_bytes, void* out, void* stream) {
    if (T < 0 || k <= 0 || E <= 0 || E > 1024 || H <= 0 || I <= 0) return W4A8_EINVAL;
    if (I % 16 || (fmt != W4A8_MX_FP4 && fmt != W4A8_MX_FP8)) return W4A8_EINVAL;
    if (H > MX_MAX_K || I > MX_MAX_N / 2 || (long long)T * k > MX_MAX_ROWS) return W4A8_EUNSUPPORTED;
    int st = mx_check_weights(2 * I, H);
    if (st || (st = mx_check_weights(H, I))) return st;
    if (T == 0) return W4A8_OK;
    if (!X || !ids || !w || !ws || !out || !aligned_to(X, 2) || !aligned_to(out, 2)) return W4A8_EINVAL;
    const int chunks = (H + 1023) / 1024, ldy = (H + 3) & ~3;
    if ((long long)T * chunks >= (1ll << 24)) return W4A8_EUNSUPPORTED;     // less than 2^32 work-items
    const MxLayerWs L = mx_layer_ws(T, k, H, I, E, fmt);
    if (ws_bytes < L.total) return W4A8_ESIZE;
    if (!aligned_to(ws, 256)) return W4A8_EINVAL;
    uint8_t* b = static_cast<uint8_t*>(ws);
    uint8_t *xq = b + L.xq, *sx = b + L.sx, *hq = b + L.hq, *sh = b + L.sh;
    int32_t *rows = reinterpret_cast<int32_t*>(b + L.rows), *offs = reinterpret_cast<int32_t*>(b + L.offs),
            *inv = reinterpret_cast<int32_t*>(b + L.inv);
    const int R = T * k;
    if ((st = check_mx(xq, sx, fmt, rows, k, offs, E, R, T, gu, gu_stride, H, 2 * I))) return st;
    if ((st = check_mx(hq, sh, fmt, nullptr, k, offs, E, R, R, dn, d_stride, I, H))) return st;
    // every step's checks have passed: from here on only a launch error can stop the chain
    if ((st = w4a8_mx_quant(X, W4A8_BF16, T, H, H, fmt, xq, sx, stream))) return st;
    if ((st = w4a8_moe_align(ids, T, k, E, rows, offs, inv, stream))) return st;
    if ((st = w4a8_moe_gemm_silu_mx_quant(xq, sx, fmt, rows, k, offs, E, R, T, gu, gu_stride, H, I, fmt, hq, sh, stream))) return st;
    // the output is bfloat16: the expert's float32 sums need not be the exact ones
    MxArgs a = mx_args(hq, sh, fmt, nullptr, k, offs, E, R, R, dn, d_stride, I, H);
    a.N = H, a.Y = b + L.yd, a.ldy = size_t(ldy), a.out = W4A8_F32;
    if ((st = run_mx("w4a8_moe_forward_mx (down)", a, fmt, false, false, I, static_cast<hipStream_t>(stream)))) return st;
    mx_combine_kernel<<<dim3(unsigned(T * chunks)), dim3(256), 0, static_cast<hipStream_t>(stream)>>>(
        reinterpret_cast<const float*>(b + L.yd), unsigned(ldy), inv, w, k, H, chunks, static_cast<uint16_t*>(out));
    return launched();
}

}  // extern "C"
