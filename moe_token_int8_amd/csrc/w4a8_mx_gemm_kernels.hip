// Products of MX activations (MXFP4 or MXFP8) with packed MXFP4 weights, dense and by expert: the streaming kernel, the launches,
// the C entry points and the expert layer.
//
// Sources (cited with the page's own section names):
//   P1 "Kimi 2.7 MoE: from 4-bit storage to INT8 (W4A8)" (pwwt.cn), section 4.4: the grouped expert GEMM and the steps of the
//      layer; section 5.1: tiles matched to the MFMA operands.
//   P3 "Quantization: formats, error and the real execution path" (wineandchord.com): FP4 / FP8 with block scales.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "w4a8_mx_gemm.h"

namespace w4a8 {

// Streaming kernel: few rows, bound by the read of the weights.
//
// A workgroup of 8 waves owns one tile of up to 16 MS rows of one expert and CT MFMA tiles of 16 weight columns (paired form:
// gate columns in half of them, the matching up columns in the others) over all of K.  The waves share the steps of 128 k: wave
// w takes w, w + 8, ...; weights and activations go from memory to registers in the layout of the MFMA operands (a step of a
// weight tile is one contiguous KiB), with no LDS and no barrier in the loop, two of a wave's steps in flight.  The 8 partial
// sums are added in wave order through LDS, so a call repeats bit for bit.
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
    constexpr int COLS = PAIR ? CT * 8 : CT * 16;
    constexpr bool QUADS = !PAIR && CT == 4;                    // the scales of the 4 tiles are one word
    constexpr int STEP_BYTES = FMT == W4A8_MX_FP4 ? 64 : 128;   // of an activation row
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, c16 = lane & 15;
    for (unsigned item = blockIdx.x;; item += gridDim.x) {
        const int slot = int(item / unsigned(ncb)), cb = int(item - unsigned(slot) * unsigned(ncb));
        const TileRows tr = mx_find<16 * MS>(a, slot, lane);
        const int expert = __builtin_amdgcn_readfirstlane(tr.expert);
        if (expert < 0) return;                                 // uniform over the workgroup; no later slot has a tile
        const int rbeg = __builtin_amdgcn_readfirstlane(tr.rbeg), nrows = __builtin_amdgcn_readfirstlane(tr.rend) - rbeg;

        // weights and their scales: descriptors that end with the expert's; tiles past the last column and steps past the last of K
        // are given an offset past them and load zeros (steps of the loop are loaded and multiplied without a branch, which
        // would cost copies of the operands; the activations of such a step are those of step 0)
        const uint8_t* wexp = a.W + size_t(expert) * a.expert_stride;
        const int width = PAIR ? 2 * a.N : a.N, ntiles = (width + 15) / 16;
        const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(wexp), 0,
                                                                            int(unsigned(ntiles) * unsigned(a.K1) * 1024u), 0x00020000);
        const __amdgpu_buffer_rsrc_t sr = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(wexp + a.scales_off), 0, int(unsigned((ntiles + 3) / 4) * unsigned(a.K1) * 256u), 0x00020000);
        constexpr unsigned NONE = 0x80000000u;                  // codes end below it, so that a sum with a valid offset does not wrap
        unsigned woff[CT], soff[QUADS ? 1 : CT];
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            const int own = PAIR ? cb * (CT / 2) + t % (CT / 2) : cb * CT + t;      // among the gate, or all, tiles
            const int tile = PAIR && t >= CT / 2 ? own + a.N / 16 : own;
            const bool there = own < (PAIR ? a.N / 16 : ntiles);
            woff[t] = there ? unsigned(tile) * unsigned(a.K1) * 1024u + unsigned(lane) * 16u : NONE;
            if (!QUADS) soff[QUADS ? 0 : t] = there ? unsigned(tile >> 2) * unsigned(a.K1) * 256u + unsigned(lane) * 4u + unsigned(tile & 3) : NONE;
        }
        if (QUADS) soff[0] = unsigned(cb) * unsigned(a.K1) * 256u + unsigned(lane) * 4u;
        struct Step {
            v4i w[CT];
            uint32_t sw[QUADS ? 1 : CT];
            MxOperand<FMT> x[MS];
            uint32_t sx[MS];
        };
        // NT: the non-temporal hint, for calls that read more weights than the Infinity Cache holds.
        auto load_w = [&](Step& b, const int step) __attribute__((always_inline)) {
            const unsigned at = step < a.K1 ? unsigned(step) * 1024u : NONE, sat = step < a.K1 ? unsigned(step) * 256u : NONE;
#pragma unroll
            for (int t = 0; t < CT; ++t)
                b.w[t] = __builtin_amdgcn_raw_buffer_load_b128(wr, woff[t] + at, 0, NT ? 2 : 0);
#pragma unroll
            for (int t = 0; t < (QUADS ? 1 : CT); ++t)
                b.sw[t] = QUADS ? uint32_t(__builtin_amdgcn_raw_buffer_load_b32(sr, soff[t] + sat, 0, 0))
                                : uint32_t(__builtin_amdgcn_raw_buffer_load_b8(sr, soff[t] + sat, 0, 0));
        };
        const uint8_t* xrow[MS];
        const uint8_t* srow[MS];
        auto load_x = [&](Step& b, const int s) __attribute__((always_inline)) {
            const int step = s < a.K1 ? s : 0;
#pragma unroll
            for (int ms = 0; ms < MS; ++ms) {
                const uint8_t* p = xrow[ms] + unsigned(step) * unsigned(STEP_BYTES);
                b.x[ms].p[0] = *reinterpret_cast<const v4i*>(p);
                if constexpr (FMT != W4A8_MX_FP4) b.x[ms].p[1] = *reinterpret_cast<const v4i*>(p + 64);
                b.sx[ms] = srow[ms][unsigned(step) * 4u];
            }
        };
        Step s0, s1;
        load_w(s0, wave);
        load_w(s1, wave + MXS_WAVES);
        // activation rows of this lane; rows past the tile repeat its first row (their sums are not stored)
#pragma unroll
        for (int ms = 0; ms < MS; ++ms) {
            const int row = ms * 16 + c16, src = mx_src(a, rbeg + (row < nrows ? row : 0));
            const size_t r = size_t(src < 0 ? 0 : src);
            xrow[ms] = a.X + r * a.rowb + unsigned(q) * 16u;
            srow[ms] = a.sx + r * (size_t(a.K1) * 4) + unsigned(q);
        }
        load_x(s0, wave);
        load_x(s1, wave + MXS_WAVES);

        v4f acc[CT][MS];
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int ms = 0; ms < MS; ++ms) acc[t][ms] = v4f{};
        auto multiply = [&](const Step& b) __attribute__((always_inline)) {
#pragma unroll
            for (int ms = 0; ms < MS; ++ms) {
                if constexpr (QUADS) {
                    acc[0][ms] = mx_mfma<FMT, 0>(b.w[0], b.x[ms], acc[0][ms], b.sw[0], b.sx[ms]);
                    acc[1][ms] = mx_mfma<FMT, 1>(b.w[1], b.x[ms], acc[1][ms], b.sw[0], b.sx[ms]);
                    acc[2][ms] = mx_mfma<FMT, 2>(b.w[2], b.x[ms], acc[2][ms], b.sw[0], b.sx[ms]);
                    acc[3][ms] = mx_mfma<FMT, 3>(b.w[3], b.x[ms], acc[3][ms], b.sw[0], b.sx[ms]);
                } else {
#pragma unroll
                    for (int t = 0; t < CT; ++t) acc[t][ms] = mx_mfma<FMT, 0>(b.w[t], b.x[ms], acc[t][ms], b.sw[t], b.sx[ms]);
                }
            }
        };
        for (int s = wave; s < a.K1; s += 2 * MXS_WAVES) {
            multiply(s0);
            load_w(s0, s + 2 * MXS_WAVES);
            load_x(s0, s + 2 * MXS_WAVES);
            multiply(s1);
            load_w(s1, s + 3 * MXS_WAVES);
            load_x(s1, s + 3 * MXS_WAVES);
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
                        for (int k = 0; k < 4; ++k) h[k] = mx_silu(g[k]) * u[k];
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
                for (int k = 0; k < 4; ++k) y[k] = mx_silu(y[k]) * up[k];
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

// Which kernel a call takes: the least of five estimates, in us.  The host knows rows and E, not the experts' rows: of E experts
// about E (1 - exp(-rows / E)) have any, and each ends in a row tile that is half empty.  Streaming tiles: 512 workgroups at a time
// take o and l a step.  MFMA tiles: `per` workgroups share a compute unit, a step takes l, or thr for each of them.  Either reads
// the weights at bw TB/s.  Fitted to 282 shapes (dense 1 .. 8192 rows, 8 .. 256 experts of 0.1 .. 1024 rows, K 768 .. 14336), of
// which the choice loses 5 % in the mean against the best of all, 38 % at worst.  Measured, us, streams of 16 and 32 rows / tiles of
// 32 / 64 / 256 rows: 16 x 4096 x 14336 fp8 9.0, 9.9 / 19.6 / 19.0 / 27.7; 128 x 14336 x 4096 fp4 26, 21 / 40 / 45 / 58; 2 rows for each
// of 256 experts, 2048 x 7168 fp8 397, 335 / 278 / 277 / 374; 64 rows for each of 64, 4096 x 2816 fp8 299, 254 / 133 / 125 / 135;
// 8192 x 4096 x 14336 fp4 257 with 256 rows.
enum MxKernel { MXK_STREAM16, MXK_STREAM32, MXK_TILE32, MXK_TILE64, MXK_TILE256, MXK_KERNELS };

static MxKernel choose_mx(const MxArgs& a, bool fp4, bool pair) {
    struct Rate {
        int rows, cols, per;
        double o, l, thr, bw;
    };
    static const Rate rates[2][MXK_KERNELS] = {
        {{16, 64, 2, 6.3, 0.098, 0, 4.1}, {32, 64, 2, 5.2, 0.196, 0, 3.8}, {32, 256, 4, 1.2, 0.43, 0.41, 5.1}, {64, 256, 3, 1.1, 0.47, 0.475, 4.8}, {256, 256, 1, 6.0, 0.73, 0, 3.8}},
        {{16, 64, 2, 5.6, 0.079, 0, 3.9}, {32, 64, 2, 4.1, 0.151, 0, 3.9}, {32, 256, 4, 1.0, 0.12, 0.31, 5.2}, {64, 256, 3, 1.7, 0.14, 0.35, 4.9}, {256, 256, 1, 5.9, 0.54, 0, 4.3}}};
    const double rows = a.rows, E = a.E, width = pair ? 2.0 * a.N : a.N, steps = a.K1;
    const double active = E > 1 ? std::min(rows, E * (1 - std::exp(-rows / E))) : 1;
    const double bytes = active * width * steps * 68;           // 128 k of a column
    MxKernel best = MXK_STREAM16;
    double least = 1e300;
    for (int v = 0; v < MXK_KERNELS; ++v) {
        const Rate& r = rates[fp4][v];
        const double rt = E > 1 ? std::max(active, rows / r.rows + 0.5 * active) : std::ceil(rows / r.rows), n = rt * std::ceil(width / r.cols);
        double us;
        if (v <= MXK_STREAM32) {
            us = std::max(1.0, n / 512) * (r.o + r.l * steps);
        } else {
            const double co = n / 256, full = co / r.per;
            const double rounds = full < 1 ? 1 : full < 4 ? std::ceil(full) : full + 0.5;
            us = 4 + rounds * (r.o + steps * std::max(r.l, r.thr * std::min(std::max(co, 1.0), double(r.per))));
        }
        us = std::max(us, 4 + bytes / (r.bw * 1e6));
        if (us < least) least = us, best = MxKernel(v);
    }
    return best;
}

template <int FMT, bool PAIR>
static const char* launch_mx(MxArgs a, hipStream_t s) {
    const long long rows = a.rows, E = a.E;
    a.lo = 1, a.hi = 0x7fffffff;
    // the tile kernel reaches activation rows through 32-bit offsets from X (gathered) or from its tile's first row
    const bool near = !a.gather || (long long)a.src_rows * a.rowb < 0xe0000000ll;
    const MxKernel v = choose_mx(a, FMT == W4A8_MX_FP4, PAIR);
    if (v == MXK_STREAM16) {
        launch_stream_t<FMT, PAIR, 1, 4, false>(a, rows / 16 + std::min(E, rows), s);
        return "mx_stream_kernel (16-row tiles)";
    }
    if (v == MXK_STREAM32 || !near) {
        launch_stream_t<FMT, PAIR, 2, 4, false>(a, rows / 32 + std::min(E, rows), s);
        return "mx_stream_kernel (32-row tiles)";
    }
    launch_mx_tile(a, FMT, PAIR, v == MXK_TILE32 ? MX_TILE_32 : v == MXK_TILE64 ? MX_TILE_64 : MX_TILE_256, s);
    return v == MXK_TILE32 ? "mx_tile_kernel (32 x 256)" : v == MXK_TILE64 ? "mx_tile_kernel (64 x 256)" : "mx_tile_kernel (256 x 256)";
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
