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
#include <cmath>
#include <cstdio>
#include <cstring>

#include "w4a8_internal.h"
#include "w4a8_moe_grouped.h"

namespace w4a8 {

// Streaming kernel: experts with few rows, bound by the read of their weights.
//
// A workgroup of 8 waves owns one tile of up to 16 * MS routed rows of one expert and CT MFMA tiles of 16 weight columns
// (the paired form: gate columns in half of them, the matching up columns in the others) over all of K.  The waves share K:
// wave w takes the 128-byte units w, w + 8, w + 16, ... of every row, so that at any time the workgroup reads 1 KiB runs of
// each weight row (16 KiB runs of a packed tile), and no operand is used by two waves: weights and activations go from
// memory to registers in the layout of the MFMA operands, with no LDS and no barrier in the loop.  One unit of 2 CT + 2 MS
// loads is in flight per wave; the loads of the other waves cover its wait (two units a wave take the registers of half of
// them: 64-token 256-expert 16-bit down product 1.05 against 1.01 ms).  At the end the 8 partial sums are added in wave
// order through LDS (int32 sums exactly).
constexpr int GS_WAVES = 8;

// Loads of the weights.  A load of a wave is 64 pieces of 16 bytes, and an MFMA wants one of each of 16 columns at 4 places
// along K; which places is free, as long as the activations have the same.  The loads are arranged to cover whole pieces of
// memory (with 16 of every 32 bytes in a load, the 256-expert steps read 3.7 TB/s instead of 6.6):
//  - packed codes (byte 64 h' + 16 q' of column c at (16 q' + c) * 32 + 16 h'): load h takes the quarters q' = 2 h, 2 h + 1
//    with both their halves, a contiguous KiB;
//  - row-major weights: load h takes the whole 128-byte lines of columns 8 h .. 8 h + 7, lane (q, i) the chunk 2 q + i / 8 of
//    column 8 h + i % 8.  Exchanging 8 lanes of the two loads in every 16 (pair_up) then gives chunk 2 q of all 16 columns in
//    one register set and chunk 2 q + 1 in the other.  (Loads of 64 bytes of 16 rows read 5.6 TB/s: they cannot carry
//    the non-temporal hint, which lets the other half of each line go before it is asked for.)
// unit_byte: the byte of a unit that lane group q then multiplies with in step h.
template <int FMT>
__device__ __forceinline__ unsigned unit_byte(int q, int h) {
    return FMT == GF_I8 ? unsigned(64 * (q & 1) + 32 * h + 16 * (q >> 1)) : unsigned(32 * q + 16 * h);
}

template <int FMT>
__device__ __forceinline__ void pair_up(v4i& a, v4i& b) {
    if constexpr (FMT != GF_I8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int x = a[k], y = b[k];                       // row_ror:8 into the upper, into the lower 8 of every 16 lanes
            a[k] = __builtin_amdgcn_update_dpp(x, y, 0x128, 0xF, 0xC, false);
            b[k] = __builtin_amdgcn_update_dpp(y, x, 0x128, 0xF, 0x3, false);
        }
    }
}

// The slot-th tile of MT rows over the experts served by this launch, in expert order; every wave finds it alone.  expert is
// -1 past the last tile.  The offsets of 256 experts are requested together, and the row range comes from the lane that
// loaded it: one trip to memory for up to 256 experts.
template <int MT>
__device__ __forceinline__ TileRows grouped_find(const GroupedArgs& a, int slot, int lane) {
    TileRows tr{0, 0, -1};
    int base = 0;
    for (int c0 = 0; c0 < a.E; c0 += 256) {
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
__global__ __launch_bounds__(512, 4) void moe_grouped_stream_kernel(GroupedArgs a, int ncb) {
    using acc_t = typename GroupedAcc<FMT>::type;
    constexpr int COLS = PAIR ? CT * 8 : CT * 16;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, c16 = lane & 15;
    const int units = (a.kb + 127) / 128;
    for (unsigned item = blockIdx.x;; item += gridDim.x) {
        const int slot = int(item / unsigned(ncb)), cb = int(item - unsigned(slot) * unsigned(ncb));
        const TileRows tr = grouped_find<16 * MS>(a, slot, lane);
        const int expert = __builtin_amdgcn_readfirstlane(tr.expert);
        if (expert < 0) return;                                 // uniform over the workgroup; no later slot has a tile
        const int rbeg = __builtin_amdgcn_readfirstlane(tr.rbeg), nrows = __builtin_amdgcn_readfirstlane(tr.rend) - rbeg;

        // weights: one buffer descriptor that ends with the last byte this workgroup may read (paired form: one for the
        // gate and one for the up rows); offsets past it load zeros
        const uint8_t* wexp = a.W + size_t(expert) * a.expert_stride;
        __amdgpu_buffer_rsrc_t wr[PAIR ? 2 : 1];
        unsigned woff[CT][FMT == GF_I8 ? 1 : 2];                // of this lane in each tile (and load)
        constexpr unsigned NONE = 0x7ffffff0u;
        if constexpr (FMT == GF_I8) {
            const int tile0 = cb * CT, ntiles = (a.N + 15) / 16;
            const unsigned tile_bytes = unsigned(units) * 2048u;
            wr[0] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(wexp + a.codes_off + size_t(tile0) * tile_bytes), 0,
                                                      int(unsigned(min(CT, ntiles - tile0)) * tile_bytes), 0x00020000);
#pragma unroll
            for (int t = 0; t < CT; ++t)
                woff[t][0] = tile0 + t < ntiles ? t * tile_bytes + unsigned((q >> 1) * 16 + c16) * 32u + (q & 1) * 16u : NONE;
        } else {
            const int n0 = cb * COLS, nvalid = min(COLS, a.N - n0);
            const unsigned extent = unsigned(nvalid - 1) * a.ldw + unsigned(a.kb);
#pragma unroll
            for (int p = 0; p < (PAIR ? 2 : 1); ++p)
                wr[p] = __builtin_amdgcn_make_buffer_rsrc(
                    const_cast<uint8_t*>(wexp + (size_t(n0) + (p ? size_t(a.N) : 0)) * a.ldw), 0, int(extent), 0x00020000);
#pragma unroll
            for (int t = 0; t < CT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int col = (PAIR ? t % (CT / 2) : t) * 16 + 8 * h + (c16 & 7);
                    woff[t][h] = col < nvalid ? unsigned(col) * a.ldw : NONE;
                }
        }
        const uint8_t* xrow[MS];
        v4i wv[CT][2], xv[MS][2];
        // NT: the non-temporal hint, for calls that read more weights than the Infinity Cache holds.
        auto load_w = [&](const int u) __attribute__((always_inline)) {
#pragma unroll
            for (int t = 0; t < CT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    unsigned off = NONE;
                    if constexpr (FMT == GF_I8) {
                        if (u < units && woff[t][0] != NONE) off = woff[t][0] + unsigned(u) * 2048u + 1024u * h;
                    } else {
                        const unsigned b = unsigned(u) * 128u + unsigned(2 * q + (c16 >> 3)) * 16u;
                        if (b < unsigned(a.kb) && woff[t][h] != NONE) off = woff[t][h] + b;
                    }
                    wv[t][h] = __builtin_amdgcn_raw_buffer_load_b128(wr[PAIR ? t / (CT / 2) : 0], off, 0, NT ? 2 : 0);
                }
        };
        auto load_x = [&](const int u) __attribute__((always_inline)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const unsigned b = unsigned(u) * 128u + unit_byte<FMT>(q, h);
#pragma unroll
                for (int ms = 0; ms < MS; ++ms)
                    xv[ms][h] = *reinterpret_cast<const v4i*>(xrow[ms] + (b < unsigned(a.kb) ? b : 0u));
            }
        };
        // activation rows of this lane; rows past the tile repeat its first row (their sums are not stored)
        int src[MS];
#pragma unroll
        for (int ms = 0; ms < MS; ++ms) {
            const int row = ms * 16 + c16;
            src[ms] = grouped_src(a, rbeg + (row < nrows ? row : 0));
        }
        load_w(wave);
#pragma unroll
        for (int ms = 0; ms < MS; ++ms) xrow[ms] = a.X + size_t(src[ms] < 0 ? 0 : src[ms]) * size_t(a.ldx);
        load_x(wave);

        acc_t acc[CT][MS];
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int ms = 0; ms < MS; ++ms) acc[t][ms] = acc_t{};
        for (int u = wave; u < units; u += GS_WAVES) {
#pragma unroll
            for (int t = 0; t < CT; ++t) pair_up<FMT>(wv[t][0], wv[t][1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // 16-bit values past the end of K: the weights are zero, and the activations have to be, since the bytes
                // loaded in their place may hold an infinity or a NaN
                const bool in = FMT == GF_I8 || unsigned(u) * 128u + unit_byte<FMT>(q, h) < unsigned(a.kb);
#pragma unroll
                for (int ms = 0; ms < MS; ++ms) {
                    v4i x = xv[ms][h];
                    if constexpr (FMT != GF_I8) x = in ? x : v4i{0, 0, 0, 0};
#pragma unroll
                    for (int t = 0; t < CT; ++t) acc[t][ms] = grouped_mfma<FMT>(wv[t][h], x, acc[t][ms]);
                }
            }
            load_w(u + GS_WAVES);
            load_x(u + GS_WAVES);
        }

        // the 8 partial sums: planes of 16 bytes a lane, [wave][tile][row block][lane]
        acc_t* red = reinterpret_cast<acc_t*>(smem);
        constexpr int ITEMS = CT * MS * 64, OUT = PAIR ? ITEMS / 2 : ITEMS;
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int ms = 0; ms < MS; ++ms) red[wave * ITEMS + (t * MS + ms) * 64 + lane] = acc[t][ms];
        // source rows and scales of this thread's outputs, in flight across the barrier
        constexpr int PER = (OUT + 511) / 512;
        int osrc[PER];
        float osx[PER];
        float4 osw[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int o = tid + i * 512, l = o & 63, row = ((o >> 6) % MS) * 16 + (l & 15);
            const int col = cb * COLS + ((o >> 6) / MS) * 16 + 4 * (l >> 4);
            osrc[i] = grouped_src(a, rbeg + (row < nrows ? row : 0));
            if constexpr (FMT == GF_I8) {
                osx[i] = osrc[i] < 0 ? -0.0f : a.sx[osrc[i]];     // -0: no row, as in the tile kernel
                osw[i] = *reinterpret_cast<const float4*>(wexp + a.scales_off + size_t(min(col, (a.N - 1) & ~3)) * 4);
            }
        }
        lds_barrier();
        auto total = [&](const int o) __attribute__((always_inline)) {
            acc_t s = red[o];
#pragma unroll
            for (int w = 1; w < GS_WAVES; ++w) s += red[w * ITEMS + o];
            return s;
        };
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int o = tid + i * 512, l = o & 63, row = ((o >> 6) % MS) * 16 + (l & 15);
            const int col = cb * COLS + ((o >> 6) / MS) * 16 + 4 * (l >> 4);
            if (o >= OUT || row >= nrows || col >= a.N) continue;
            const acc_t s = total(o);
            float y[4];
            if constexpr (FMT == GF_I8) {
                y[0] = (float(s[0]) * osw[i].x) * osx[i];
                y[1] = (float(s[1]) * osw[i].y) * osx[i];
                y[2] = (float(s[2]) * osw[i].z) * osx[i];
                y[3] = (float(s[3]) * osw[i].w) * osx[i];
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = __float_as_uint(osx[i]) == 0x80000000u ? 0.0f : y[k];
            } else if constexpr (PAIR) {
                const acc_t up = total(o + ITEMS / 2);
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = osrc[i] < 0 ? 0.0f : silu_gate(s[k]) * up[k];
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = osrc[i] < 0 ? 0.0f : s[k];
            }
            grouped_store(a, size_t(rbeg + row) * a.ldy + col, min(4, a.N - col), y[0], y[1], y[2], y[3]);
        }
        if constexpr (MS == 1) return;                          // one tile a workgroup
        lds_barrier();                                          // the planes are written again by the next tile
    }
}

// Workgroups of a launch over `slots` row tiles: all tiles of the 16-row class; 32-row tiles go round in a grid that is
// resident at once, two workgroups a compute unit (with one for each tile 3614 tokens of 161 experts lose 20 %, and 256
// experts of 7168 columns took 16 us to find nothing).
constexpr long long GS_GRID = 512;

template <int FMT, bool PAIR, int MS, int CT, bool NT>
static void launch_stream_t(const GroupedArgs& a, long long slots, hipStream_t s) {
    constexpr size_t lds = size_t(GS_WAVES) * CT * MS * 64 * 16;
    static_assert(lds <= 65536, "two workgroups share a compute unit");
    constexpr int cols = PAIR ? CT * 8 : CT * 16;
    const int ncb = (a.N + cols - 1) / cols;
    const long long blocks = MS == 1 ? slots * ncb : std::min(slots * ncb, GS_GRID);
    moe_grouped_stream_kernel<FMT, PAIR, MS, CT, NT><<<dim3(unsigned(blocks)), dim3(512), lds, s>>>(a, ncb);
}

// Rows that an expert has at most in a call whose tokens go to k different experts each (k as the gather has it; without a
// sensible k, all rows).  The launches are chosen by it; experts with more rows, of calls that name an expert twice for a
// token, are handled all the same.
static long long usual_most(const GroupedArgs& a) {
    return a.topk >= 1 && a.topk <= a.E ? (a.rows + a.topk - 1) / a.topk : a.rows;
}

// Whether one launch of 32-row streaming tiles over every expert beats the launches by row class.  The estimates, in us, use
// what the host knows (an upper bound of the tiles; rows / E for the rows of an expert) and rates fitted to some 300
// measured calls: 512 workgroups at a time take 1.5 to 3 us for a 32 x 64 tile, by its rows, and a nanosecond for 30 (16
// bit) or 36 bytes of its operands, all of them together 5.6 TB/s of weights; the 16-row class reads 6.7 TB/s, and its
// workgroups, some 768 at a time, take 1.9 us and 1 for 585 bytes of K; a launch costs 5 or 6; few tokens name 0.6 of the
// experts that they could.  Examples (one launch / by class): 330 tokens x 4 of 72 experts, K = 1240, I = 370: 38 / 82 us;
// 205 x 4 of 6, K = 2432, N = 897 in 8 bits: 19 / 43; 2814 x 5 of 68, K = 744, I = 19: 15 / 36; 9 x 8 of 72, K = 232,
// I = 1683: 24 / 35; 10 x 7 of 241, K = 816, I = 1764: 35 / 54; 6288 x 2 of 134, K = 3176, N = 739: 329 / 223; 2913 x 7 of
// 40, K = 384, N = 413 in 8 bits: 37 / 28; 33 x 6 of 64, K = 4096, I = 1408: 261 / 214.
static bool one_launch(const GroupedArgs& a, bool i8, bool pair) {
    const double rows = a.rows, E = a.E, avg = rows / E, kb = a.kb, width = pair ? 2.0 * a.N : a.N;
    const double most = double(usual_most(a)), experts = std::min(E, rows);
    const double weights = experts * width * kb * (most <= 64 ? 0.6 : 1.0);
    const double items = (std::floor(rows / 32) + experts) * std::ceil(width / 64);
    const double item = 1.5 + 1.5 * std::min(1.0, avg / 32) + (64 + std::min(32.0, avg)) * kb / (i8 ? 36e3 : 30e3);
    const double tiles32 = std::max(1.0, items / 512) * item;
    const double one = 6 + std::max(tiles32, weights / 5.6e6);
    double split;
    if (most <= 64) {
        const double wgs = pair ? experts * std::ceil(a.N / 16.0) : experts * std::ceil(a.N / (experts * a.N / 64 < 1024 ? 32.0 : 64.0));
        const double small = std::max(weights / 6.7e6, wgs / 768 * (1.9 + kb / 585));
        const double more = most <= 16 ? 0.0 : std::min(1.0, avg / 32);     // of the work in experts with more than 16 rows
        split = (most <= 16 ? 6 : 11) + small * (1 - more) + tiles32 * more;
    } else {
        split = (avg >= 128 ? 13 : 20) + choose_tiles(a, i8, pair).us * std::min(1.0, avg / 32) +
                weights / 6.7e6 * std::max(0.0, 1 - avg / 128);
    }
    return one < split;
}

// Row classes, one launch each: up to 16 rows, up to 64 (tiles of 32) and the MFMA tiles.  Classes that no expert of an
// ordinary call is in are left out, and the last one that is there takes all larger experts (33 tokens x 6 of 64: a launch
// that finds nothing is 5 of 214 us).  `slots` bounds the row tiles of a class.  Where experts have 128 rows on average, few
// have less than 65: those share the second launch.  Returns the kernels' names for the log.
template <int FMT, bool PAIR>
static const char* launch_grouped(GroupedArgs a, hipStream_t s) {
    const long long rows = a.rows, E = a.E, most = usual_most(a);
    constexpr int ALL = 0x7fffffff;
    // the MFMA-tile kernel reaches activation rows through 32-bit offsets from X (gathered) or from its tile's first row
    constexpr long long REACH = 0xe0000000ll;
    const bool near = a.ldx <= (1 << 23) && a.kb <= (1 << 23) && (!a.gather || (long long)a.src_rows * a.ldx < REACH);
    // a launch has less than 2^32 work-items; the 16-row class has a workgroup of 512 for each of its tiles, of 16 columns or
    // more (1024 experts of 131071 columns: 8192 tiles each, the last one short of a column, are 2^32)
    const long long slots = std::min(E, rows) + (most <= 16 ? rows / 16 : 0);
    const bool wide = slots * ((a.N + 15) / 16) >= (1ll << 23);
    if (rows > 16 && (!near || wide || one_launch(a, FMT == GF_I8, PAIR))) {
        a.lo = 1, a.hi = ALL;
        launch_stream_t<FMT, PAIR, 2, 4, false>(a, rows / 32 + std::min(E, rows), s);
        return "moe_grouped_stream_kernel (32-row tiles)";
    }
    const bool few_small = rows >= 128 * E;
    if (!few_small) {
        a.lo = 1, a.hi = most <= 16 ? ALL : 17;
        // non-temporal reads where the call's weights cannot be found in the 256 MiB Infinity Cache by the next one: 6.4 GB
        // of codes 1.09 -> 0.96 ms, but 69 MB 17.6 -> 19.5 us
        const bool nt = std::min(E, rows) * (long long)a.N * (PAIR ? 2 : 1) * a.kb > (256ll << 20);
        // column tiles of a workgroup: 4, or 2 where there are few workgroups to spread over the chip (a single token's 69 MB:
        // 17.5 -> 15.4 us; 64-token steps of 256 experts lose 4 %) and in the paired form (33 tokens: 240 -> 225 us)
        const long long blocks = slots * ((a.N + 63) / 64);
        if constexpr (PAIR) {
            if (nt) launch_stream_t<FMT, PAIR, 1, 2, true>(a, slots, s);
            else launch_stream_t<FMT, PAIR, 1, 2, false>(a, slots, s);
        } else {
            if (nt) launch_stream_t<FMT, PAIR, 1, 4, true>(a, slots, s);
            else if (blocks < 1024) launch_stream_t<FMT, PAIR, 1, 2, false>(a, slots, s);
            else launch_stream_t<FMT, PAIR, 1, 4, false>(a, slots, s);
        }
        if (most <= 16) return "moe_grouped_stream_kernel (16-row tiles)";
    }
    a.lo = few_small ? 1 : 17, a.hi = most <= 64 ? ALL : 65;
    launch_stream_t<FMT, PAIR, 2, 4, false>(a, rows / 32 + std::min(E, rows / a.lo), s);
    if (most <= 64) return "moe_grouped_stream_kernel (by rows)";
    a.lo = 65, a.hi = ALL;
    return launch_grouped_tile(a, FMT, PAIR, s) ? "moe_grouped_stream_kernel (by rows), moe_grouped_tile_kernel (128 x 128)"
                                                : "moe_grouped_stream_kernel (by rows), moe_grouped_tile_kernel (256 x 256)";
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static int launched() { return hipGetLastError() == hipSuccess ? W4A8_OK : W4A8_EHIP; }

// Columns a launch may have: 16 rows of as many experts make 2^20 workgroups.
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
    const char* names = launch_grouped<GF_I8, false>(a, s);
    if (log_on())
        std::fprintf(stderr, "w4a8: w4a8_moe_gemm_w8a8 E=%d rows=%d K=%d N=%d -> %s\n", E, rows, L.K, L.N, names);
    return launched();
}

static int run_w16(const void* X, int dtype, int ldx, const int32_t* gather, int k, const int32_t* offsets, int E, int rows,
                   int src_rows, const void* W, size_t stride, int ldw, int K, int N, bool pair, void* Y, int ldy,
                   int out_dtype, hipStream_t s) {
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
    const char* names = dtype == W4A8_BF16 ? (pair ? launch_grouped<GF_BF16, true>(a, s) : launch_grouped<GF_BF16, false>(a, s))
                                           : (pair ? launch_grouped<GF_F16, true>(a, s) : launch_grouped<GF_F16, false>(a, s));
    if (log_on())
        std::fprintf(stderr, "w4a8: w4a8_moe_gemm%s_w16a16 E=%d rows=%d K=%d N=%d %s -> %s\n", pair ? "_silu" : "", E, rows, K,
                     N, dtype == W4A8_F16 ? "float16" : "bfloat16", names);
    return launched();
}

static size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace of a layer: pieces in order, each 256-byte aligned.  The W8A8 layer has the pieces and sizes of
// w4a8_moe_workspace_size; the W16A16 layer the routing, h and the expert outputs.
struct LayerWs {
    size_t xq = 0, sx = 0, rows = 0, offs = 0, inv = 0, gu = 0, hq = 0, sh = 0, yd = 0, total = 0;
};

static LayerWs layer_ws(int T, int k, int H, int I, int E, bool w8) {
    const size_t R = size_t(T) * size_t(k);
    LayerWs w;
    size_t o = 0;
    auto piece = [&](size_t bytes) {
        const size_t at = o;
        o = align256(o + bytes);
        return at;
    };
    if (w8) w.xq = piece(size_t(T) * H), w.sx = piece(size_t(T) * 4);
    w.rows = piece(R * 4);
    w.offs = piece(size_t(E + 1) * 4);
    w.inv = piece(R * 4);
    w.gu = piece(R * size_t(I) * (w8 ? 4 : 2));                 // gate and up, or h
    if (w8) w.hq = piece(R * size_t(I)), w.sh = piece(R * 4);
    w.yd = piece(R * size_t(H) * 2);
    w.total = o;
    return w;
}

static int layer_check(const void* X, const int32_t* ids, const float* w, int T, int k, int E, const void* ws, size_t ws_bytes,
                size_t need, const void* out) {
    if (T < 0 || k <= 0 || E <= 0 || E > 1024) return W4A8_EINVAL;
    if ((long long)T * k > GROUPED_MAX_ROWS) return W4A8_EUNSUPPORTED;
    if (T == 0) return W4A8_OK;
    if (!X || !ids || !w || !ws || !out || !aligned16(X) || !aligned16(out)) return W4A8_EINVAL;
    if (ws_bytes < need) return W4A8_ESIZE;
    return (reinterpret_cast<uintptr_t>(ws) & 255u) ? W4A8_EINVAL : W4A8_OK;
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

size_t w4a8_moe_w16a16_workspace_size(int T, int k, int H, int I, int E) {
    if (T < 0 || k <= 0 || H <= 0 || I <= 0 || E <= 0) return 0;
    return layer_ws(T, k, H, I, E, false).total;
}

int w4a8_moe_forward_w8a8(const void* X, const int32_t* ids, const float* w, int T, int k, int E, const void* gu_blobs,
                          size_t gu_stride, const w4a8_wdesc* gu_desc, const void* d_blobs, size_t d_stride,
                          const w4a8_wdesc* d_desc, void* ws, size_t ws_bytes, void* out, void* stream) {
    int st = check_w8(gu_desc);
    if (st || (st = check_w8(d_desc))) return st;
    const int H = gu_desc->K, I = gu_desc->N / 2;
    if (gu_desc->N % 2 || d_desc->K != I || d_desc->N != H) return W4A8_EINVAL;
    if (T < 0 || k <= 0 || E <= 0) return W4A8_EINVAL;
    if (H > 65536 || I > 16384) return W4A8_EUNSUPPORTED;       // rows of the two quantizations
    const LayerWs L = layer_ws(T, k, H, I, E, true);
    if ((st = layer_check(X, ids, w, T, k, E, ws, ws_bytes, L.total, out)) || T == 0) return st;
    uint8_t* b = static_cast<uint8_t*>(ws);
    int8_t *xq = reinterpret_cast<int8_t*>(b + L.xq), *hq = reinterpret_cast<int8_t*>(b + L.hq);
    float *sx = reinterpret_cast<float*>(b + L.sx), *sh = reinterpret_cast<float*>(b + L.sh);
    int32_t *rows = reinterpret_cast<int32_t*>(b + L.rows), *offs = reinterpret_cast<int32_t*>(b + L.offs),
            *inv = reinterpret_cast<int32_t*>(b + L.inv);
    const int R = T * k;
    if ((st = check_w8_call(xq, sx, rows, k, offs, E, R, T, gu_blobs, gu_stride, gu_desc, b + L.gu, W4A8_BF16))) return st;
    if ((st = check_w8_call(hq, sh, nullptr, k, offs, E, R, R, d_blobs, d_stride, d_desc, b + L.yd, W4A8_BF16))) return st;
    // every step's checks have passed: from here on only a launch error can stop the chain
    hipStream_t s = static_cast<hipStream_t>(stream);
    if ((st = w4a8_quant_act(X, T, H, H, xq, sx, stream))) return st;
    if ((st = w4a8_moe_align(ids, T, k, E, rows, offs, inv, stream))) return st;
    if ((st = run_w8(xq, sx, rows, k, offs, E, R, T, gu_blobs, gu_stride, gu_desc, b + L.gu, W4A8_BF16, s))) return st;
    if ((st = w4a8_silu_mul_quant(b + L.gu, R, I, hq, sh, stream))) return st;
    if ((st = run_w8(hq, sh, nullptr, k, offs, E, R, R, d_blobs, d_stride, d_desc, b + L.yd, W4A8_BF16, s))) return st;
    return w4a8_moe_combine(b + L.yd, inv, w, T, k, H, out, stream);
}

int w4a8_moe_forward_w16a16(const void* X, const int32_t* ids, const float* w, int T, int k, int E, const void* Wgu,
                            size_t gu_stride, const void* Wd, size_t d_stride, int H, int I, void* ws, size_t ws_bytes,
                            void* out, void* stream) {
    if (T < 0 || k <= 0 || E <= 0 || H <= 0 || I <= 0) return W4A8_EINVAL;
    const LayerWs L = layer_ws(T, k, H, I, E, false);
    int st = layer_check(X, ids, w, T, k, E, ws, ws_bytes, L.total, out);
    if (st || T == 0) return st;
    uint8_t* b = static_cast<uint8_t*>(ws);
    int32_t *rows = reinterpret_cast<int32_t*>(b + L.rows), *offs = reinterpret_cast<int32_t*>(b + L.offs),
            *inv = reinterpret_cast<int32_t*>(b + L.inv);
    const int R = T * k, dt = W4A8_BF16;
    if ((st = check_w16_call(X, dt, H, rows, k, offs, E, R, T, Wgu, gu_stride, H, H, I, true, b + L.gu, I, dt))) return st;
    if ((st = check_w16_call(b + L.gu, dt, I, nullptr, k, offs, E, R, R, Wd, d_stride, I, I, H, false, b + L.yd, H, dt)))
        return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if ((st = w4a8_moe_align(ids, T, k, E, rows, offs, inv, stream))) return st;
    if ((st = run_w16(X, dt, H, rows, k, offs, E, R, T, Wgu, gu_stride, H, H, I, true, b + L.gu, I, dt, s))) return st;
    if ((st = run_w16(b + L.gu, dt, I, nullptr, k, offs, E, R, R, Wd, d_stride, I, I, H, false, b + L.yd, H, dt, s))) return st;
    return w4a8_moe_combine(b + L.yd, inv, w, T, k, H, out, stream);
}

}  // extern "C"
