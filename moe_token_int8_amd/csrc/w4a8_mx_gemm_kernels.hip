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

// Streaming kernel: few rows, bound by the read of the weights and, in small calls, by its latency.
//
// A workgroup of 8 waves owns one tile of up to 16 rows of one expert and 4 MFMA tiles of 16 weight columns (paired form: 2 of gate
// columns, then the 2 matching ones of up columns) over all of K.  The waves share the steps of 128 k: wave w takes w, w + 8, ...;
// weights and activations go from memory to registers in the layout of the MFMA operands (a step of a weight tile is one
// contiguous KiB), with no LDS and no barrier in the loop, two of a wave's steps in flight.  The 8 partial sums are added in wave
// order through LDS, so a call repeats bit for bit.  8 x 4096 x 14336 in fp8: 8.5 us (31 MB: 5 at the rate of a large read); one token's
// 6 experts, 4096 x 1408 gate/up: 12.9 (37 MB: 6), of which the loads of activations take 1.4 us and the second MFMA of a step 1.
// (Two row tiles a workgroup read the weights once for 32 rows, but the tile kernel does that faster: 32 rows for each of 64
// experts, 1408 x 4096 fp4 73 against 51 us.  Three steps in flight: 9.7 in place of 8.4.)
constexpr int MXS_WAVES = 8, MXS_ROWS = 16, MXS_TILES = 4;

// The slot-th row tile over the experts, in their order; every wave finds it alone.  expert is -1 past the last one.
__device__ __forceinline__ TileRows mx_find(const MxArgs& a, int slot, int lane) {
    TileRows tr{0, 0, -1};
    if (!a.offsets) {
        if ((long long)slot * MXS_ROWS < a.rows) tr = {slot * MXS_ROWS, min(a.rows, slot * MXS_ROWS + MXS_ROWS), 0};
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
            if (c0 + j * 64 >= a.E) break;
            // malformed offsets cannot move a tile outside the rows of the call
            const int e0 = min(max(b[j], 0), a.rows), e1 = min(max(e[j], e0), a.rows), cnt = e1 - e0;
            const int t = (cnt + MXS_ROWS - 1) / MXS_ROWS;
            const int incl = wave_prefix(t);
            const unsigned long long hit = __ballot(slot >= base + incl - t && slot < base + incl);
            if (hit) {
                const int src = __ffsll((long long)hit) - 1;
                tr.expert = c0 + j * 64 + src;
                tr.rbeg = __builtin_amdgcn_readlane(e0 + (slot - base - (incl - t)) * MXS_ROWS, src);
                tr.rend = min(__builtin_amdgcn_readlane(e1, src), tr.rbeg + MXS_ROWS);
                return tr;
            }
            base += __builtin_amdgcn_readlane(incl, 63);
        }
    }
    return tr;
}

template <int FMT, bool PAIR>
__global__ __launch_bounds__(512, 4) void mx_stream_kernel(MxArgs a, int ncb, int slots) {
    constexpr int CT = MXS_TILES, COLS = PAIR ? CT * 8 : CT * 16;
    constexpr int STEP_BYTES = FMT == W4A8_MX_FP4 ? 64 : 128;   // of an activation row
    __shared__ v4f red[MXS_WAVES * CT * 64];                    // partial sums: [wave][tile][lane]
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, c16 = lane & 15;
    const int first = int(blockIdx.x / unsigned(ncb)), cb = int(blockIdx.x - unsigned(first) * unsigned(ncb));
    for (int slot = first; slot < slots; slot += int(gridDim.x / unsigned(ncb))) {
        const TileRows tr = mx_find(a, slot, lane);
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
        unsigned woff[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            const int own = PAIR ? cb * (CT / 2) + t % (CT / 2) : cb * CT + t;      // among the gate, or all, tiles
            const int tile = PAIR && t >= CT / 2 ? own + a.N / 16 : own;
            const bool there = own < (PAIR ? a.N / 16 : ntiles);
            woff[t] = there ? unsigned(tile) * unsigned(a.K1) * 1024u + unsigned(lane) * 16u : NONE;
        }
        // the scales of the 4 tiles are one word (paired form: see MxPairScales)
        const MxPairScales ps = mx_pair_scales<NONE>(a, cb * 2, cb * 2 < a.N / 16, lane);
        const unsigned soff = unsigned(cb) * unsigned(a.K1) * 256u + unsigned(lane) * 4u;
        struct Step {
            v4i w[CT];
            uint32_t sw[PAIR ? 3 : 1];
            MxOperand<FMT> x;
            uint32_t sx;
        };
        auto load_w = [&](Step& b, const int step) __attribute__((always_inline)) {
            const unsigned at = step < a.K1 ? unsigned(step) * 1024u : NONE, sat = step < a.K1 ? unsigned(step) * 256u : NONE;
#pragma unroll
            for (int t = 0; t < CT; ++t) b.w[t] = __builtin_amdgcn_raw_buffer_load_b128(wr, woff[t] + at, 0, 0);
            b.sw[0] = uint32_t(__builtin_amdgcn_raw_buffer_load_b32(sr, (PAIR ? ps.gate : soff) + sat, 0, 0));
            if constexpr (PAIR) {
                b.sw[1] = uint32_t(__builtin_amdgcn_raw_buffer_load_b32(sr, ps.up + sat, 0, 0));
                b.sw[2] = uint32_t(__builtin_amdgcn_raw_buffer_load_b32(sr, ps.up2 + sat, 0, 0));
            }
        };
        const uint8_t *xrow, *srow;
        auto load_x = [&](Step& b, const int s) __attribute__((always_inline)) {
            const int step = s < a.K1 ? s : 0;
            const uint8_t* p = xrow + unsigned(step) * unsigned(STEP_BYTES);
            b.x.p[0] = *reinterpret_cast<const v4i*>(p);
            if constexpr (FMT != W4A8_MX_FP4) b.x.p[1] = *reinterpret_cast<const v4i*>(p + 64);
            b.sx = srow[unsigned(step) * 4u];
        };
        Step s0, s1;
        load_w(s0, wave);
        load_w(s1, wave + MXS_WAVES);
        // the activation row of this lane; rows past the tile repeat its first row (their sums are not stored)
        const int src = mx_src(a, rbeg + (c16 < nrows ? c16 : 0));
        {
            const size_t r = size_t(src < 0 ? 0 : src);
            xrow = a.X + r * a.rowb + unsigned(q) * 16u;
            srow = a.sx + r * (size_t(a.K1) * 4) + unsigned(q);
        }
        load_x(s0, wave);
        load_x(s1, wave + MXS_WAVES);

        v4f acc[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t) acc[t] = v4f{};
        auto multiply = [&](const Step& b) __attribute__((always_inline)) {
            if constexpr (PAIR) {
                const uint32_t g = b.sw[0] >> ps.gshift, u = __builtin_amdgcn_alignbyte(b.sw[2], b.sw[1], ps.ubyte);
                acc[0] = mx_mfma<FMT, 0>(b.w[0], b.x, acc[0], g, b.sx);
                acc[1] = mx_mfma<FMT, 1>(b.w[1], b.x, acc[1], g, b.sx);
                acc[2] = mx_mfma<FMT, 0>(b.w[2], b.x, acc[2], u, b.sx);
                acc[3] = mx_mfma<FMT, 1>(b.w[3], b.x, acc[3], u, b.sx);
            } else {
                acc[0] = mx_mfma<FMT, 0>(b.w[0], b.x, acc[0], b.sw[0], b.sx);
                acc[1] = mx_mfma<FMT, 1>(b.w[1], b.x, acc[1], b.sw[0], b.sx);
                acc[2] = mx_mfma<FMT, 2>(b.w[2], b.x, acc[2], b.sw[0], b.sx);
                acc[3] = mx_mfma<FMT, 3>(b.w[3], b.x, acc[3], b.sw[0], b.sx);
            }
        };
        // (fp8 pairs: loads held back until the operands of the step before are free; moved ahead of them they spilled registers, 256 rows
        // of 64 experts, 4096 x 1408 gate/up, 86 us in place of 71.  Unpaired, held back, 512 tokens x 6 of 64, 1408 x 4096,
        // 141 in place of 117)
        for (int s = wave; s < a.K1; s += 2 * MXS_WAVES) {
            multiply(s0);
            if constexpr (PAIR && FMT != W4A8_MX_FP4) __builtin_amdgcn_sched_barrier(0);
            load_w(s0, s + 2 * MXS_WAVES);
            load_x(s0, s + 2 * MXS_WAVES);
            multiply(s1);
            if constexpr (PAIR && FMT != W4A8_MX_FP4) __builtin_amdgcn_sched_barrier(0);
            load_w(s1, s + 3 * MXS_WAVES);
            load_x(s1, s + 3 * MXS_WAVES);
        }

        constexpr int ITEMS = CT * 64, OUT = PAIR ? ITEMS / 2 : ITEMS;
#pragma unroll
        for (int t = 0; t < CT; ++t) red[wave * ITEMS + t * 64 + lane] = acc[t];
        lds_barrier();
        auto total = [&](const int o) __attribute__((always_inline)) {
            v4f s = red[o];
#pragma unroll
            for (int w = 1; w < MXS_WAVES; ++w) s += red[w * ITEMS + o];
            return s;
        };
        if (tid < OUT) {                                        // whole waves
            if (PAIR && a.Hq) {                                 // 8 neighbouring lanes take a row's block of 32 columns
                const int j = tid & 7, row = tid >> 3, at = (j >> 2) * 64 + (j & 3) * 16 + row, block = cb * (COLS / 32);
                v4f h{};
                const bool dead = __shfl(src, row & 15, 64) < 0;
                if (row < nrows && cb * COLS + j * 4 < a.N && !dead) {
                    const v4f g = total(at), u = total(at + ITEMS / 2);
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[k] = mx_silu(g[k]) * u[k];
                }
                mx_store_block(a, rbeg + row, block, j, h, row < nrows);
                if (row < nrows && cb * COLS + COLS >= a.N) mx_pad_blocks(a, rbeg + row, block + 1, j);
            } else {
                const int row = c16, col = cb * COLS + (tid >> 6) * 16 + 4 * q;
                if (row < nrows && col < a.N) {
                    v4f y = total(tid);
                    if constexpr (PAIR) {
                        const v4f up = total(tid + ITEMS / 2);
#pragma unroll
                        for (int k = 0; k < 4; ++k) y[k] = mx_silu(y[k]) * up[k];
                    }
                    if (src < 0) y = v4f{};
                    mx_store(a, size_t(rbeg + row) * a.ldy + col, min(4, a.N - col), y);
                }
            }
        }
        lds_barrier();                                          // the sums are written again by the next tile
    }
}

// A workgroup for each tile, up to a number that keeps a launch's work-items below 2^32; beyond it they go round.
template <int FMT, bool PAIR>
static void launch_stream(const MxArgs& a, hipStream_t s) {
    constexpr int cols = PAIR ? MXS_TILES * 8 : MXS_TILES * 16;
    const int ncb = (a.N + cols - 1) / cols;                    // at most 2^14
    const int slots = a.rows / MXS_ROWS + std::min(a.E, a.rows);                // an upper bound of the row tiles
    mx_stream_kernel<FMT, PAIR><<<dim3(unsigned(std::min(slots, (1 << 22) / ncb) * ncb)), dim3(512), 0, s>>>(a, ncb, slots);
}

// Which kernel a call takes: the least of six estimates, in us.  The host knows rows and E, not the experts' rows: of E experts
// about E (1 - exp(-rows / E)) have any, and each ends in a row tile that is half empty.  n tiles meet c n / 256 times on a compute
// unit (c > 1: a launch that fits does not spread evenly).  Streaming tiles, two of which share a unit, take o and l a step.  Of MFMA
// tiles `per` share one, a step takes l, or thr for each of them.  Either reads the weights at bw TB/s, which adds up with the steps as
// far as a norm of third powers says.  Fitted to 414 shapes for fp4 and 243 for fp8 (dense 1 .. 8192 rows, 8 .. 256 experts of 0.1 ..
// 1024 rows, evenly or skewed, K 300 .. 14336), of which the choice loses 2 % (fp8 1.3) in the mean against the best of all, 27 %
// (fp8 20) at worst; an fp8 step has twice the MFMAs of an fp4 one.  Measured, us, fp8, streaming / tiles of 32 x 128, 32 x 256, 64 x
// 256, 128 x 256 and 128 x 512:
//   16 x 4096 x 14336                      9 /  20,  23,  33,  57,  78       128 x 4096 x 14336            36 /  27,  26,  35,  58,  80
//   256 x 14336 x 4096                     - /  65,  67, 101, 182, 253       2048 x 14336 x 4096            - / 186, 183, 162, 253, 258
//   2048 x 4096 x 14336                    - / 201, 207, 185, 176, 173
//   4 rows for each of 256, 2048 x 7168  405 / 326, 333, 379, 566, 573       64 rows for each, the same     - / 682, 633, 598, 730, 737
enum MxKernel { MXK_STREAM, MXK_SMALL, MXK_TILE32, MXK_TILE64, MXK_TILE128, MXK_WIDE, MXK_KERNELS };

static MxKernel choose_mx(const MxArgs& a, int N, bool fp4, bool pair, MxKernel first) {
    struct Rate {
        int rows, cols, per;
        double o, l, thr, bw, c;
    };
    static const Rate rates[2][MXK_KERNELS] = {{{16, 64, 2, 2.30, 0.163, 0.000, 6.80, 1.67}, {32, 128, 4, 1.78, 0.449, 0.254, 6.35, 1.83},
                                                {32, 256, 4, 0.93, 0.560, 0.513, 5.95, 1.22}, {64, 256, 2, 3.07, 0.006, 0.749, 6.14, 2.00},
                                                {128, 256, 2, 3.57, 1.884, 1.278, 6.58, 1.44}, {128, 512, 1, 5.74, 0.032, 2.388, 7.57, 1.99}},
                                               {{16, 64, 2, 1.55, 0.108, 0.000, 7.80, 2.00}, {32, 128, 4, 0.00, 0.196, 0.171, 5.43, 1.46},
                                                {32, 256, 4, 0.00, 0.275, 0.301, 5.69, 1.33}, {64, 256, 2, 1.81, 0.106, 0.301, 5.40, 1.71},
                                                {128, 256, 2, 3.40, 0.195, 0.446, 6.00, 1.73}, {128, 512, 1, 5.24, 0.351, 0.803, 6.04, 2.00}}};
    const double rows = a.rows, E = a.E, width = pair ? 2.0 * N : N, steps = a.K1;
    const double active = E > 1 ? std::min(rows, E * (1 - std::exp(-rows / E))) : 1;
    const double bytes = active * width * steps * 68;           // 128 k of a column
    MxKernel best = first;
    double least = 1e300;
    for (int v = first; v < MXK_KERNELS; ++v) {
        const Rate& r = rates[fp4][v];
        const double rt = E > 1 ? std::max(active, rows / r.rows + 0.5 * active) : std::ceil(rows / r.rows);
        const double n = rt * std::ceil(width / r.cols);
        double us;
        if (v == MXK_STREAM) {
            us = std::max(1.0, r.c * n / 512) * (r.o + r.l * steps);
        } else {
            const double co = n / 256, full = co / r.per;
            const double rounds = full < 1 ? 1 : full < 4 ? std::ceil(full) : full + 0.5;
            us = 4 + rounds * (r.o + steps * std::max(r.l, r.thr * std::min(std::max(r.c * co, 1.0), double(r.per))));
        }
        const double read = 4 + bytes / (r.bw * 1e6);
        us = std::cbrt(us * us * us + read * read * read);
        if (us < least) least = us, best = MxKernel(v);
    }
    return best;
}

// N: columns of the whole product, of which a.N may be a slice.  A slice streams where the whole would, since that sums in another order
// than tiles do (all of which sum alike): its bits are those of the whole.
template <int FMT, bool PAIR>
static const char* launch_mx(const MxArgs& a, int N, hipStream_t s) {
    // the tile kernel reaches activation rows through 32-bit offsets from X (gathered) or from its tile's first row
    const bool near = !a.gather || (long long)a.src_rows * a.rowb < 0xe0000000ll, fp4 = FMT == W4A8_MX_FP4;
    MxKernel kernel = near ? choose_mx(a, N, fp4, PAIR, MXK_STREAM) : MXK_STREAM;
    if (kernel != MXK_STREAM && a.N != N) kernel = choose_mx(a, a.N, fp4, PAIR, MXK_SMALL);
    switch (kernel) {
        case MXK_SMALL: launch_mx_tile(a, FMT, PAIR, MX_TILE_SMALL, s); return "mx_tile_kernel (32 x 128)";
        case MXK_TILE32: launch_mx_tile(a, FMT, PAIR, MX_TILE_32, s); return "mx_tile_kernel (32 x 256)";
        case MXK_TILE64: launch_mx_tile(a, FMT, PAIR, MX_TILE_64, s); return "mx_tile_kernel (64 x 256)";
        case MXK_TILE128: launch_mx_tile(a, FMT, PAIR, MX_TILE_128, s); return "mx_tile_kernel (128 x 256)";
        case MXK_WIDE: launch_mx_tile(a, FMT, PAIR, MX_TILE_WIDE, s); return "mx_tile_kernel (128 x 512)";
        default: launch_stream<FMT, PAIR>(a, s); return "mx_stream_kernel";
    }
}

// out[t] = sum_j w[t, j] Yd[inv[t, j]] in float32, j ascending, rounded once: the experts' outputs stay in float32 (rounded to
// bfloat16 in between, a layer's error against float64 is 2.5e-3 normwise in place of 1.7e-3, that of the one rounding).
// 4 columns a thread; the rows of 8 experts are requested together.  N columns (a slice of out, whose rows have ldo).
__global__ __launch_bounds__(256) void mx_combine_kernel(const float* Yd, unsigned ldy, const int32_t* inv, const float* w, int k, int N,
                                                         int chunks, uint16_t* out, unsigned ldo) {
    const int t = int(blockIdx.x / unsigned(chunks)), c = (int(blockIdx.x % unsigned(chunks)) * 256 + int(threadIdx.x)) * 4;
    if (c >= N) return;
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
    uint16_t* p = out + size_t(t) * ldo + c;
    if (c + 4 <= N) {
        *reinterpret_cast<u2*>(p) = u2{f32_to_bf16_pair(s[0], s[1]), f32_to_bf16_pair(s[2], s[3])};
    } else {
        for (int i = 0; i < N - c; ++i) p[i] = uint16_t(f32_to_bf16_rne(s[i]));
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
    // the tile kernel numbers its tiles, of 32 rows (and one more for each expert) by 64 columns of the weights or larger, in 32 bits
    if ((long long)(rows / 32 + E) * ((width + 63) / 64) >= (1ll << 32)) return W4A8_EUNSUPPORTED;
    if (rows == 0) return W4A8_OK;
    if (!Xq || !sx || !W || (E > 1 && !offsets)) return W4A8_EINVAL;
    if (gather ? (k <= 0 || src_rows == 0) : src_rows < rows) return W4A8_EINVAL;
    if (E > 1 && stride < mx_layout(width, K).total) return W4A8_EINVAL;
    if (!aligned_to(Xq, 16) || !aligned_to(sx, 4) || !aligned_to(W, 16) || (stride & 15)) return W4A8_EINVAL;
    if (!aligned_to(gather, 4) || !aligned_to(offsets, 4)) return W4A8_EINVAL;
    return W4A8_OK;
}

static int check_out(const void* Y, int ldy, int N, int out, bool f32) {
    if (out != W4A8_BF16 && out != W4A8_F16 && !(f32 && out == W4A8_F32)) return W4A8_EINVAL;
    if (ldy < N || !Y || !aligned_to(Y, out == W4A8_F32 ? 4 : 2)) return W4A8_EINVAL;
    return W4A8_OK;
}

// Sizes of a layer.
static int check_layer(int T, int k, int H, int I, int E, int fmt) {
    if (T < 0 || k <= 0 || E <= 0 || E > 1024 || H <= 0 || I <= 0) return W4A8_EINVAL;
    if (I % 16 || (fmt != W4A8_MX_FP4 && fmt != W4A8_MX_FP8)) return W4A8_EINVAL;
    if (H > MX_MAX_K || I > MX_MAX_N / 2 || (long long)T * k > MX_MAX_ROWS) return W4A8_EUNSUPPORTED;
    if ((long long)T * ((H + 1023) / 1024) >= (1ll << 24)) return W4A8_EUNSUPPORTED;    // work-items of the sum: less than 2^32
    const int st = mx_check_weights(2 * I, H);
    return st ? st : mx_check_weights(H, I);
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
    // s = ceil(log2 k), 2^32 (2^s - k) / k + 1: exact for dividends below 2^32, of which the sum takes those below 2^31
    while ((1ll << a.div_shift) < k) ++a.div_shift;
    a.div_mul = gather ? unsigned(((1ull << 32) * ((1ull << a.div_shift) - unsigned(k))) / unsigned(k) + 1) : 0;
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

// N: columns of the whole product (a.N: of this launch).
static int run_mx(const char* call, MxArgs& a, int N, int fmt, bool pair, int K, hipStream_t s) {
    const char* names = fmt == W4A8_MX_FP4 ? (pair ? launch_mx<W4A8_MX_FP4, true>(a, N, s) : launch_mx<W4A8_MX_FP4, false>(a, N, s))
                                           : (pair ? launch_mx<W4A8_MX_FP8, true>(a, N, s) : launch_mx<W4A8_MX_FP8, false>(a, N, s));
    if (log_on())
        std::fprintf(stderr, "w4a8: %s E=%d rows=%d K=%d N=%d %s -> %s\n", call, a.E, a.rows, K, a.N,
                     fmt == W4A8_MX_FP4 ? "mxfp4" : "mxfp8", names);
    return launched();
}

// Up to so many routed rows one launch makes the codes of the tokens and the order of the rows.  A whole layer of H 2048, I 1408,
// k 8, fp8, two launches against one, us: 64 experts, 1 token 22.8 / 21.2, 256 tokens 112 / 109, 512 tokens 148 / 150; 8 experts, 256
// tokens 66.3 / 65.7, 512 tokens 113 / 120.
constexpr int MX_ROUTE_ROWS = 2048;

// Workspace of the layer: pieces in order, each 256-byte aligned.
struct MxLayerWs {
    size_t xq, sx, rows, offs, inv, hq, sh, yd, total;
    int slice;                // columns of the experts' outputs that yd holds at a time
};

// The experts' float32 outputs come last and take what `bytes` leaves: all H columns where they fit, else equal slices of whole groups
// of 64, whose down products and sums follow each other (slice 0: no room for 64).  The launches of a second slice cost 8 to 14 us (H
// 4096, I 1408, 64 experts, k 6, fp4: 4 tokens 49 -> 57, 33 tokens 109 -> 124, 512 tokens 167 -> 176, skewed 161 -> 189), and prompts
// nothing; more slices gain nothing there either (8192 tokens: whole 1042, two slices 1050, four 1024, eight 1036).
static MxLayerWs mx_layer_ws(int T, int k, int H, int I, int E, int fmt, size_t bytes) {
    const size_t R = size_t(T) * size_t(k);
    MxLayerWs w;
    size_t o = 0;
    auto piece = [&](size_t size) {
        const size_t at = o;
        o = (o + size + 255) & ~size_t(255);
        return at;
    };
    w.xq = piece(size_t(T) * mx_row_bytes(fmt, H)), w.sx = piece(size_t(T) * size_t(mx_kp(H) / 32));
    w.rows = piece(R * 4), w.offs = piece(size_t(E + 1) * 4), w.inv = piece(R * 4);
    w.hq = piece(R * mx_row_bytes(fmt, I)), w.sh = piece(R * size_t(mx_kp(I) / 32));
    const size_t before = o;
    w.yd = piece(R * size_t((H + 3) & ~3) * 4);                 // float32, rows at whole 16 bytes
    w.total = o;
    w.slice = H;
    if (bytes < w.total) {
        const size_t fit = bytes < before || R == 0 ? 0 : (bytes - before) / (R * 4) / 64 * 64;
        const size_t slices = fit ? (size_t(H) + fit - 1) / fit : 0;
        w.slice = slices ? int((size_t(H) + slices - 1) / slices + 63) / 64 * 64 : 0;
    }
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
    return run_mx("w4a8_mx_gemm", a, N, fmt, false, K, static_cast<hipStream_t>(stream));
}

int w4a8_moe_gemm_mx(const void* Xq, const uint8_t* sx, int fmt, const int32_t* gather, int k, const int32_t* offsets, int E, int rows,
                     int src_rows, const void* blobs, size_t stride, int K, int N, void* Y, int ldy, int out_dtype, void* stream) {
    int st = check_mx(Xq, sx, fmt, gather, k, offsets, E, rows, src_rows, blobs, stride, K, N);
    if (st || rows == 0) return st;
    if (!offsets) return W4A8_EINVAL;
    if ((st = check_out(Y, ldy, N, out_dtype, true))) return st;
    MxArgs a = mx_args(Xq, sx, fmt, gather, k, offsets, E, rows, src_rows, blobs, stride, K, N);
    a.N = N, a.Y = Y, a.ldy = size_t(ldy), a.out = out_dtype;
    return run_mx("w4a8_moe_gemm_mx", a, N, fmt, false, K, static_cast<hipStream_t>(stream));
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
    return run_mx("w4a8_moe_gemm_silu_mx", a, I, fmt, true, K, static_cast<hipStream_t>(stream));
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
    return run_mx("w4a8_moe_gemm_silu_mx_quant", a, I, fmt, true, K, static_cast<hipStream_t>(stream));
}

size_t w4a8_moe_mx_workspace_size(int T, int k, int H, int I, int E, int fmt) {
    return check_layer(T, k, H, I, E, fmt) ? 0 : mx_layer_ws(T, k, H, I, E, fmt, ~size_t(0)).total;
}

int w4a8_moe_forward_mx(const void* X, const int32_t* ids, const float* w, int T, int k, int E, int fmt, const void* gu, size_t gu_stride,
                        const void* dn, size_t d_stride, int H, int I, void* ws, size_t ws_bytes, void* out, void* stream) {
    int st = check_layer(T, k, H, I, E, fmt);
    if (st || T == 0) return st;
    if (!X || !ids || !w || !ws || !out || !aligned_to(X, 2) || !aligned_to(out, 2) || !aligned_to(ids, 4) || !aligned_to(w, 4))
        return W4A8_EINVAL;
    const MxLayerWs L = mx_layer_ws(T, k, H, I, E, fmt, ws_bytes);
    if (L.slice == 0) return W4A8_ESIZE;
    if (!aligned_to(ws, 256)) return W4A8_EINVAL;
    uint8_t* b = static_cast<uint8_t*>(ws);
    uint8_t *xq = b + L.xq, *sx = b + L.sx, *hq = b + L.hq, *sh = b + L.sh;
    int32_t *rows = reinterpret_cast<int32_t*>(b + L.rows), *offs = reinterpret_cast<int32_t*>(b + L.offs),
            *inv = reinterpret_cast<int32_t*>(b + L.inv);
    const int R = T * k;
    if ((st = check_mx(xq, sx, fmt, rows, k, offs, E, R, T, gu, gu_stride, H, 2 * I))) return st;
    if ((st = check_mx(hq, sh, fmt, nullptr, k, offs, E, R, R, dn, d_stride, I, H))) return st;
    // every step's checks have passed: from here on only a launch error can stop the chain
    if (R <= MX_ROUTE_ROWS) {
        launch_route_quant(ids, R, E, rows, offs, inv, X, T, H, fmt, xq, sx, static_cast<hipStream_t>(stream));
        if ((st = launched())) return st;
    } else {
        if ((st = w4a8_mx_quant(X, W4A8_BF16, T, H, H, fmt, xq, sx, stream))) return st;
        if ((st = w4a8_moe_align(ids, T, k, E, rows, offs, inv, stream))) return st;
    }
    if ((st = w4a8_moe_gemm_silu_mx_quant(xq, sx, fmt, rows, k, offs, E, R, T, gu, gu_stride, H, I, fmt, hq, sh, stream))) return st;
    const int slice = L.slice, ldy = (slice + 3) & ~3;
    const MxArgs whole = mx_args(hq, sh, fmt, nullptr, k, offs, E, R, R, dn, d_stride, I, H);
    for (int c = 0; c < H; c += slice) {
        MxArgs a = whole;
        a.N = std::min(slice, H - c), a.Y = b + L.yd, a.ldy = size_t(ldy), a.out = W4A8_F32;
        a.W += size_t(c / 16) * size_t(a.K1) * 1024;            // codes by 16 columns, scales by 64
        a.scales_off = whole.scales_off - size_t(c / 16) * size_t(a.K1) * 1024 + size_t(c / 64) * size_t(a.K1) * 256;
        if ((st = run_mx("w4a8_moe_forward_mx (down)", a, H, fmt, false, I, static_cast<hipStream_t>(stream)))) return st;
        const int chunks = (a.N + 1023) / 1024;
        mx_combine_kernel<<<dim3(unsigned(T * chunks)), dim3(256), 0, static_cast<hipStream_t>(stream)>>>(
            reinterpret_cast<const float*>(b + L.yd), unsigned(ldy), inv, w, k, a.N, chunks, static_cast<uint16_t*>(out) + c, unsigned(H));
        if ((st = launched())) return st;
    }
    return W4A8_OK;
}

}  // extern "C"
