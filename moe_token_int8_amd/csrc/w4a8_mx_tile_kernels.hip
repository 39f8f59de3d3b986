// Products of MX activations with packed MXFP4 weights: the kernel for many rows (MFMA tiles), dense and by expert.
//
// Source: P1 "Kimi 2.7 MoE: from 4-bit storage to INT8 (W4A8)" (pwwt.cn), section 4.4 step 4 (the grouped expert GEMM over
// router-sorted rows, "the performance key") and section 5.1 (tiles matched to the MFMA operands).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "w4a8_mx_gemm.h"

namespace w4a8 {

// Persistent workgroups of WN waves walk over tiles of 16 MT rows x 64 WN weight columns (paired form: half of them gate, the
// matching half up columns).  Each wave owns all rows and 64 columns: 4 MT accumulators of 4 a lane.
//
// The packed weights are in operand order, so they go from memory straight to registers, 4 KiB a wave and step of 128 k, two
// steps ahead (DEEP: five), each to one wave.  Only the activations pass through LDS: in stages of 128 bytes a row (two steps of fp4,
// one of fp8), copied without registers (buffer_load ... lds), three stages deep (DEEP, fp8: six), with a stage's scale bytes behind
// its codes.  DEEP is for launches of few tiles, whose time is one chain of steps over K, each waiting for its loads: 192 x 14336 x 4096 in
// fp4, tiles of 32 x 128: 31 -> 26 us (fp8, whose chain is one of MFMAs: 62 either way).
//
// What bounds it: in fp8 the MFMAs, two for each step of 16 x 16 (see mx_mfma; 2.2 PFLOP/s by themselves), and the split of the operands
// between them, which every wave does for all rows: MFMAs are busy for 63 % of a prompt's cycles.  8192^3 takes 653 us (1.68 PFLOP/s),
// with one MFMA, which loses small parts, 332.
// In fp4 the path of the vector memory, 64 bytes a cycle and compute unit.  A 128 x 512 step of fp4 moves 40 KiB, 640 cycles of the
// MFMAs' 1024, and each scale of a row costs a cycle.  4096 x 14336 x 4096 in fp4: 102 us (4.7 PFLOP/s; MFMAs alone on registers reach
// 6.2), 83 without the memory operations in the loop, 99 without the copies, 94 without the weights, unchanged with half the LDS
// reads.  256 x 256 tiles, where two waves load the same weights, took 108; touching the weights' lines 8 steps ahead, one load of
// 64 lines, 115 to 130 (64 cycles of the same path); another order of steps for workgroups that share data, no change.
//
// vmcnt counts in the order of issue, so what is issued when is fixed: a step requests the weights of the step AHEAD steps on; the
// first step of a stage then requests the activations of the stage NST - 1 stages on.  One barrier a stage, before the last
// group of MFMAs, when the stage's last operands are in registers: behind it the next stage is whole and this one is free.
constexpr int MXT_ROW = 128;                                    // bytes of a row in a stage
constexpr int MXT_MAX_E = 1024;
constexpr unsigned MXT_PANEL = 8;                               // row tiles of a panel of consecutive tiles

#define LDS __attribute__((address_space(3)))
using lds_ptr = LDS uint8_t*;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_buffer(const uint8_t* base, size_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, int(unsigned(bytes < 0xffffffffu ? bytes : 0xffffffffu)),
                                             0x00020000);
}

// 16 or 4 bytes a lane from memory to LDS, lane after lane from dst on.  (The whole offset is in the register operand: a scalar
// offset is not part of the range check.)
__device__ __forceinline__ void mx_copy16(__amdgpu_buffer_rsrc_t src, unsigned off, lds_ptr dst) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (LDS void*)dst, 16, off, 0, 0, 0);
}
__device__ __forceinline__ void mx_copy4(__amdgpu_buffer_rsrc_t src, unsigned off, lds_ptr dst) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (LDS void*)dst, 4, off, 0, 0, 0);
}

// Waits until at most NEWER memory operations of this wave are in flight and its LDS reads are done, then for every wave.
template <int NEWER>
__device__ __forceinline__ void mx_barrier() {
    static_assert(NEWER < 64, "the counter has 6 bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((NEWER & 15) | ((NEWER >> 4) << 14) | (7 << 4) | (0 << 8));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// v, without what the compiler knows of it: what is derived from it is computed there and not kept across the MFMA loop.
__device__ __forceinline__ int mx_opaque(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// Chunk c (16 bytes) of row r sits at position c ^ mx_swizzle(r): 16 rows read at one chunk lie in distinct banks.
__device__ __forceinline__ int mx_swizzle(int r) { return (r >> 1) & 7; }

// Exchanges the odd 16-lane rows of a with the even ones of b.
__device__ __forceinline__ void mx_swap16(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0], b = r[1];
}
// Maximum over the four lanes l % 16, 16 + l % 16, ...
__device__ __forceinline__ uint32_t mx_max_rows(uint32_t m) {
    const auto a = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max(uint32_t(a[0]), uint32_t(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return max(uint32_t(b[0]), uint32_t(b[1]));
}

template <int FMT, bool PAIR, int WN, int MT, bool DEEP>
__global__ __launch_bounds__(64 * WN, MT == 8 || DEEP ? 2 : FMT != W4A8_MX_FP4 ? 3 : 4)
void mx_tile_kernel(MxArgs a) {
    constexpr bool FP4 = FMT == W4A8_MX_FP4;
    constexpr int THREADS = 64 * WN, BM = 16 * MT;
    constexpr int COLS = PAIR ? 32 * WN : 64 * WN;              // columns of Y
    constexpr int SPS = FP4 ? 2 : 1;                            // steps of a stage
    constexpr int CODES = BM * MXT_ROW, STAGE = CODES + THREADS * 4;
    constexpr int SETS = DEEP ? 6 : 3, AHEAD = SETS - 1;        // register sets of weights, steps that they are requested ahead
    constexpr int NST = DEEP && !FP4 ? 6 : 3;                   // stages of activations
    constexpr int SB = 4 * SPS;                                 // scale bytes of a row in a stage
    constexpr int COPIES = BM * 8 / THREADS;                    // 16-byte copies of a thread in a stage
    constexpr int G = FP4 ? MT / 2 : MT == 8 ? 2 : 1, NG = MT / G;      // row tiles of a group, groups of a step
    constexpr int FILL = COPIES + 1, WL = PAIR ? 7 : 5;         // memory operations of a stage's copies, of a step's weights
    constexpr int LIST = 64;                                    // tiles looked up at a time
    static_assert(NG % 2 == 0 && COPIES * THREADS == BM * 8 && BM * SB <= THREADS * 4, "shapes");
    __shared__ __align__(1024) uint8_t stage0[STAGE];
    __shared__ __align__(1024) uint8_t stage1[STAGE];
    __shared__ __align__(1024) uint8_t stage2[STAGE];
    __shared__ __align__(1024) uint8_t stage3[NST > 3 ? STAGE : 16];
    __shared__ __align__(1024) uint8_t stage4[NST > 3 ? STAGE : 16];
    __shared__ __align__(1024) uint8_t stage5[NST > 3 ? STAGE : 16];
    __shared__ int4 list[LIST];                                 // tiles of this workgroup: expert, first row, rows, column block
    __shared__ int first[MXT_MAX_E + 1];                        // row tiles before expert e
    __shared__ int entries[(BM + 63) / 64 * 64];                // gather entries of the next tile's rows: a whole wave's copy at a time
    __shared__ int wsum[WN];
    const int lane = int(threadIdx.x) & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int q = lane >> 4, c16 = lane & 15, wn = wave;
    const int ncb = (a.N + COLS - 1) / COLS;
    const int stages = (a.K1 + SPS - 1) / SPS;
    const bool f32 = !PAIR && a.out == W4A8_F32;

    // row tiles of every expert, as a prefix sum
    {
        constexpr int EPT = MXT_MAX_E / THREADS;
        const int tid = threadIdx.x;
        int t[EPT], incl = 0;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const int e = EPT * tid + i;
            const int cnt = e < a.E ? max(mx_row_last(a, e) - mx_row_first(a, e), 0) : 0;
            t[i] = (cnt + BM - 1) / BM;
            incl += t[i];
        }
        int excl = -incl;
        incl = wave_prefix(incl);
        if (lane == 63) wsum[wave] = incl;
        __syncthreads();
        for (int w = 0; w < wave; ++w) incl += wsum[w];
        excl += incl;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            if (EPT * tid + i <= a.E) first[EPT * tid + i] = excl;
            excl += t[i];
        }
        if (a.E == MXT_MAX_E && tid == THREADS - 1) first[MXT_MAX_E] = incl;
        __syncthreads();
    }
    // Workgroups take the tiles in turn.  Within an expert, panels of MXT_PANEL row tiles go through all columns together.  (The calls
    // refuse what has 2^32 tiles or more.)  Consecutive tiles for a workgroup, which keep its weights from one to the next, share less
    // in L2: 4153 tokens x 6 of 64 experts, 4096 x 2815 320 us in place of 270.
    const unsigned total = unsigned(first[a.E]) * unsigned(ncb);
    // blocks go to the 8 XCDs in turn: the blocks of one XCD take neighbouring tiles, which share rows or columns in its L2
    const unsigned nblk = gridDim.x, per = nblk / 8;
    const unsigned rank = nblk % 8 ? blockIdx.x : blockIdx.x % 8 * per + blockIdx.x / 8;
    const int mine = rank < total ? int((total - rank - 1) / nblk + 1) : 0;         // tiles of this workgroup
    if (mine == 0) return;

    // the tiles from k0 on of this workgroup; all threads, between barriers
    auto look_up = [&](const int k0) __attribute__((always_inline)) {
        const int tid = mx_opaque(int(threadIdx.x));
        if (tid < LIST && k0 + tid < mine) {
            const unsigned t = rank + unsigned(k0 + tid) * nblk, trow = t / unsigned(ncb);
            int lo = 0, hi = a.E;                               // expert: the last one whose first tile is not after trow
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (unsigned(first[mid]) <= trow) lo = mid;
                else hi = mid;
            }
            const unsigned in_e = t - unsigned(first[lo]) * unsigned(ncb), panel = in_e / (MXT_PANEL * unsigned(ncb));
            const unsigned j = in_e - panel * (MXT_PANEL * unsigned(ncb));
            const unsigned rp = min(MXT_PANEL, unsigned(first[lo + 1] - first[lo]) - panel * MXT_PANEL);
            const int cb = int(j / rp), r0 = mx_row_first(a, lo) + int(panel * MXT_PANEL + j - unsigned(cb) * rp) * BM;
            list[tid] = make_int4(lo, r0, min(BM, mx_row_last(a, lo) - r0), cb);
        }
        __syncthreads();
    };

    // What a tile reads.  Descriptors end with the data: rows past the tile's last and weight tiles past the last column are given
    // an offset past everything and load zeros.  The step goes into the weights' scalar offset, which the range check leaves
    // out: steps past the last one, which are requested but not used, repeat it.
    constexpr unsigned NONE = 0xf0000000u;
    unsigned xoff[COPIES], soff, woff[4], wsoff = NONE;
    MxPairScales ps{NONE, NONE, NONE, 0, 0};                    // paired form
    __amdgpu_buffer_rsrc_t xr, sr, wr, wsr;
    v4i w[SETS][4];
    uint32_t sw[SETS][PAIR ? 3 : 1];

    auto load_w_part = [&](const int set, const int step, const int part) __attribute__((always_inline)) {
        const int k = min(step, a.K1 - 1);
        if (part < 4) w[set][part & 3] = __builtin_amdgcn_raw_buffer_load_b128(wr, woff[part & 3], k * 1024, 0);
        else sw[set][PAIR ? part - 4 : 0] = uint32_t(__builtin_amdgcn_raw_buffer_load_b32(
                 wsr, !PAIR ? wsoff : part == 4 ? ps.gate : part == 5 ? ps.up : ps.up2, k * 256, 0));
    };
    auto load_w = [&](const int set, const int step) __attribute__((always_inline)) {
#pragma unroll
        for (int part = 0; part < WL; ++part) load_w_part(set, step, part);
    };
    auto copy_part = [&](const lds_ptr st, const int s, const int part) __attribute__((always_inline)) {
        const bool in = s < stages;
        if (part < COPIES)
            mx_copy16(xr, xoff[part < COPIES ? part : 0] + (in ? unsigned(s) * MXT_ROW : 0xc0000000u),
                      st + (part * (THREADS / 8) + wave * 8) * MXT_ROW);
        else
            mx_copy4(sr, soff + (in ? unsigned(s) * SB : 0xc0000000u), st + CODES + wave * 256);
    };
    auto copies = [&](const lds_ptr st, const int s) __attribute__((always_inline)) {
#pragma unroll
        for (int part = 0; part < FILL; ++part) copy_part(st, s, part);
    };
    const lds_ptr sts[6] = {(lds_ptr)stage0, (lds_ptr)stage1, (lds_ptr)stage2, (lds_ptr)stage3, (lds_ptr)stage4, (lds_ptr)stage5};

    // gather entries of a tile's rows, copied to LDS a tile ahead
    auto request_rows = [&](const int4 g) __attribute__((always_inline)) {
        if (a.gather && wave < (BM + 63) / 64)
            mx_copy4(mx_buffer(reinterpret_cast<const uint8_t*>(a.gather + g.y), size_t(g.z) * 4),
                     unsigned(mx_opaque(int(threadIdx.x))) * 4u, (lds_ptr)((LDS int*)entries + wave * 64));
    };
    auto source = [&](const int g) __attribute__((always_inline)) {    // row of X, or -1
        return a.gather ? mx_token(a, g) : g;
    };
    // bit m of dead: this lane's row 16 m + c16 of the wave has a gather entry that names no row (its outputs are zeros)
    unsigned dead = 0, next_dead = 0;
    auto begin = [&](const int4 g) __attribute__((always_inline)) {
        const int tid = mx_opaque(int(threadIdx.x)), lane = tid & 63;
        const uint8_t* wexp = a.W + size_t(g.x) * a.expert_stride;
        const int width = PAIR ? 2 * a.N : a.N, ntiles = (width + 15) / 16;
        wr = mx_buffer(wexp, size_t(ntiles) * size_t(a.K1) * 1024);
        wsr = mx_buffer(wexp + a.scales_off, size_t((ntiles + 3) / 4) * size_t(a.K1) * 256);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int own = PAIR ? g.w * 2 * WN + wn * 2 + (n & 1) : g.w * 4 * WN + wn * 4 + n;  // among the gate, or all, tiles
            const int t = PAIR && n >= 2 ? own + a.N / 16 : own;
            const bool there = own < (PAIR ? a.N / 16 : ntiles);
            woff[n] = there ? unsigned(t) * (unsigned(a.K1) * 1024u) + unsigned(lane) * 16u : NONE;
        }
        if (PAIR) {
            const int tile = (g.w * WN + wn) * 2;
            ps = mx_pair_scales<NONE>(a, tile, tile < a.N / 16, lane);
        } else {
            const int quad = g.w * WN + wn;
            wsoff = quad * 4 < ntiles ? unsigned(quad) * (unsigned(a.K1) * 256u) + unsigned(lane) * 4u : NONE;
        }
        const size_t srow = size_t(a.K1) * 4, base = a.gather ? 0 : size_t(g.y), nrow = size_t(a.gather ? a.src_rows : g.z);
        xr = mx_buffer(a.X + base * a.rowb, nrow * a.rowb);
        sr = mx_buffer(a.sx + base * srow, nrow * srow);
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const int row = i * (THREADS / 8) + (tid >> 3), chunk = (lane & 7) ^ mx_swizzle(row);
            const int src = max(source(a.gather ? entries[row] : row), 0);
            xoff[i] = row < g.z ? unsigned(src) * a.rowb + unsigned(chunk) * 16u : NONE;
        }
        {
            const int row = FP4 ? tid >> 1 : tid;
            const int src = row < BM ? max(source(a.gather ? entries[min(row, BM - 1)] : row), 0) : 0;
            soff = row < g.z ? unsigned(src) * unsigned(srow) + (FP4 ? unsigned(tid & 1) * 4u : 0u) : NONE;
        }
        if (a.gather) {
            next_dead = 0;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int row = m * 16 + (lane & 15);
                if (row < g.z && source(entries[row]) < 0) next_dead |= 1u << m;
            }
        }
        // as the steps before the first one would: the waits below count on this order
#pragma unroll
        for (int t = -SPS * (NST - 1) < -AHEAD ? -SPS * (NST - 1) : -AHEAD; t < 0; ++t) {
            __builtin_amdgcn_sched_barrier(0);
            if (t + AHEAD >= 0) load_w(t + AHEAD, t + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
            if ((t + SPS * NST) % SPS == 0 && t / SPS + NST - 1 >= 0) copies(sts[t / SPS + NST - 1], t / SPS + NST - 1);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // operations behind the copies of stage 0 at the start
    constexpr int NEWER_FIRST = FP4 ? (AHEAD < 3 ? AHEAD : 3) * WL + FILL : (NST - 2) * (WL + FILL);
    // behind those of stage s + 1 at the barrier of stage s, which stands before the last group of its last step
    constexpr int OPS = FP4 ? WL : WL + FILL;                       // of that step, spread over its row tiles
    constexpr int NEWER = (FP4 ? 2 * WL + FILL : (NST - 3) * (WL + FILL)) + (MT - G) * OPS / MT;
    static_assert((NST * SPS) % SETS == 0 && (FP4 ? NST == 3 : AHEAD == NST - 1), "what the counts are made for");

    // operands in LDS: byte offsets of this lane in a stage, for the halves of 64 bytes
    int xat[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) xat[h] = mx_opaque(c16 * MXT_ROW + ((4 * h + q) ^ mx_swizzle(c16)) * 16);
    const int sat = mx_opaque(CODES + c16 * SB + q);
    MxOperand<FMT> x[2][G];
    uint32_t sx[2][G];
    auto read_tile = [&](const int buf, const lds_ptr st, const int h, const int m) __attribute__((always_inline)) {
        const int i = m % G;
        if constexpr (FP4) {
            x[buf][i].p[0] = *(const LDS v4i*)(st + xat[h] + m * 2048);
        } else {
            x[buf][i].p[0] = *(const LDS v4i*)(st + xat[0] + m * 2048);
            x[buf][i].p[FP4 ? 0 : 1] = *(const LDS v4i*)(st + xat[1] + m * 2048);
        }
        sx[buf][i] = *(const LDS uint8_t*)(st + sat + m * 16 * SB + (FP4 ? 4 * h : 0));
    };

    // Stores that a wave issues at the end of a tile, behind the next one's first copies: FEW of a regular tile in 16 bits, twice as
    // many in float32 or of quantized h, or a number that is not known (0), which the first barrier waits for.
    constexpr int FEW = PAIR ? MT : 2 * MT;
    int stores = 0;

    look_up(0);
    auto uniform = [&](int4 v) __attribute__((always_inline)) {
        return make_int4(__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y),
                         __builtin_amdgcn_readfirstlane(v.z), __builtin_amdgcn_readfirstlane(v.w));
    };
    int4 g = uniform(list[0]);
    request_rows(g);
    mx_barrier<0>();
    begin(g);
    for (int k = 0;;) {
        const int4 cur = g;
        dead = next_dead;
        if (stores == FEW) mx_barrier<NEWER_FIRST + FEW>();
        else if (stores == 2 * FEW) mx_barrier<NEWER_FIRST + 2 * FEW>();
        else mx_barrier<NEWER_FIRST>();
        // the next tile, and its gather entries: requested here, first needed at the end of this tile
        if (++k < mine) {
            if (k % LIST == 0) look_up(k);
            g = uniform(list[k % LIST]);
            request_rows(g);
        }
        {
            v4f acc[4][MT];
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[n][m] = v4f{};
#pragma unroll
            for (int m = 0; m < G; ++m) read_tile(0, sts[0], 0, m);
            for (int s0 = 0;; s0 += NST) {
#pragma unroll
                for (int u = 0; u < NST; ++u) {
                    const lds_ptr st = sts[u], next = sts[(u + 1) % NST], far = sts[(u + NST - 1) % NST];
#pragma unroll
                    for (int h = 0; h < SPS; ++h) {
                        // A step: for each row tile the operands of a row tile of the next group are read, a share of the step's memory
                        // operations is issued, and 4 MFMAs follow.  (Issued together at the start of the step, the memory operations
                        // of all waves meet: 4096 x 14336 x 4096 in fp4 113 us in place of 104.)
                        const int step = (s0 + u) * SPS + h, set = (u * SPS + h) % SETS;
                        const int ops = h == 0 ? WL + FILL : WL;
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const int gr = m / G, i = m % G, b = gr & 1;
                            const bool last = gr == NG - 1 && h == SPS - 1;
                            if (last && i == 0) mx_barrier<NEWER>();
                            if (gr < NG - 1) read_tile(b ^ 1, st, h, m + G);
                            else if (!last) read_tile(0, st, 1, i);
                            else read_tile(0, next, 0, i);
#pragma unroll
                            for (int op = m * ops / MT; op < (m + 1) * ops / MT; ++op) {
                                if (op < WL) load_w_part((set + AHEAD) % SETS, step + AHEAD, op);
                                else copy_part(far, s0 + u + NST - 1, op - WL);
                            }
                            __builtin_amdgcn_sched_barrier(0);
                            if constexpr (PAIR) {
                                if (m == 0) {                   // the bytes in place, once a step
                                    sw[set][0] >>= ps.gshift;
                                    sw[set][PAIR ? 1 : 0] = __builtin_amdgcn_alignbyte(sw[set][PAIR ? 2 : 0], sw[set][PAIR ? 1 : 0], ps.ubyte);
                                }
                                acc[0][m] = mx_mfma<FMT, 0>(w[set][0], x[b][i], acc[0][m], sw[set][0], sx[b][i]);
                                acc[1][m] = mx_mfma<FMT, 1>(w[set][1], x[b][i], acc[1][m], sw[set][0], sx[b][i]);
                                acc[2][m] = mx_mfma<FMT, 0>(w[set][2], x[b][i], acc[2][m], sw[set][PAIR ? 1 : 0], sx[b][i]);
                                acc[3][m] = mx_mfma<FMT, 1>(w[set][3], x[b][i], acc[3][m], sw[set][PAIR ? 1 : 0], sx[b][i]);
                            } else {
                                acc[0][m] = mx_mfma<FMT, 0>(w[set][0], x[b][i], acc[0][m], sw[set][0], sx[b][i]);
                                acc[1][m] = mx_mfma<FMT, 1>(w[set][1], x[b][i], acc[1][m], sw[set][0], sx[b][i]);
                                acc[2][m] = mx_mfma<FMT, 2>(w[set][2], x[b][i], acc[2][m], sw[set][0], sx[b][i]);
                                acc[3][m] = mx_mfma<FMT, 3>(w[set][3], x[b][i], acc[3][m], sw[set][0], sx[b][i]);
                            }
                            __builtin_amdgcn_sched_barrier(0);
                        }
                        if (step + 1 >= a.K1) goto done;
                    }
                }
            }
        done:;
            const int l = mx_opaque(lane), c16 = l & 15, q = l >> 4;
            // every stage has been read, and what was requested past the last step (nothing is read there) has ended: the next
            // tile's copies start before this one's outputs are stored
            mx_barrier<0>();
            if (k < mine) begin(g);
            const unsigned gone = dead;
            auto value = [&](const int n, const int m) __attribute__((always_inline)) {
                v4f y = acc[n][m];
                if constexpr (PAIR) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = mx_silu(y[i]) * acc[n + (PAIR ? 2 : 0)][m][i];
                }
                return gone >> m & 1 ? v4f{} : y;
            };
            const unsigned es = f32 ? 4u : 2u;
            const bool regular = !(PAIR && a.Hq) && a.ldy < (size_t(1) << 21) && ((a.N & (f32 ? 3 : 7)) == 0 || (cur.w + 1) * COLS <= a.N);
            const unsigned pitch = unsigned(a.ldy) * es;
            const int colw = cur.w * COLS + wn * (PAIR ? 32 : 64);  // first column of the wave
            stores = !regular ? 0 : f32 ? 2 * FEW : FEW;
            if (PAIR && a.Hq) {
                const unsigned bpr = unsigned(mx_kp(a.N) / 32), block = unsigned(colw) / 32u;
                const bool have = colw < a.N, fp4 = a.h_fmt == W4A8_MX_FP4;
                const unsigned bytes = fp4 ? 16u : 32u;
                // rows past the tile's last lie behind its descriptors: their stores are dropped
                const __amdgpu_buffer_rsrc_t hr = mx_buffer(a.Hq + size_t(cur.y) * bpr * bytes, size_t(cur.z) * bpr * bytes);
                const __amdgpu_buffer_rsrc_t br = mx_buffer(a.sh + size_t(cur.y) * bpr, size_t(cur.z) * bpr);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    v4f h0 = value(0, m), h1 = value(1, m);
                    if (colw + 16 >= a.N) h1 = v4f{};           // a last block of 16 columns
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = max(top, max(__float_as_uint(h0[i]) & 0x7fffffffu, __float_as_uint(h1[i]) & 0x7fffffffu));
                    top = mx_max_rows(top);
                    const uint32_t byte = fp4 ? mx_scale_byte<W4A8_MX_FP4>(top) : mx_scale_byte<W4A8_MX_FP8>(top);
                    const float up = byte == 255u ? 0.0f : mx_up(byte);
                    uint32_t c0, c1;
                    h0 *= up, h1 *= up;
                    if (fp4) c0 = mx_fp4x4(h0[0], h0[1], h0[2], h0[3]), c1 = mx_fp4x4(h1[0], h1[1], h1[2], h1[3]);
                    else c0 = mx_fp8x4(h0[0], h0[1], h0[2], h0[3]), c1 = mx_fp8x4(h1[0], h1[1], h1[2], h1[3]);
                    if (byte == 255u) c0 = 0u, c1 = 0u;
                    mx_swap16(c0, c1);                          // 8 neighbouring columns: tile q % 2, half q / 2
                    const unsigned at = unsigned(m * 16 + c16) * bpr + block, at8 = unsigned((q & 1) * 2 + (q >> 1));
                    if (fp4) __builtin_amdgcn_raw_buffer_store_b32(int(c0 | (c1 << 16)), hr, have ? at * 16u + at8 * 4u : NONE, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b64(v2i{int(c0), int(c1)}, hr, have ? at * 32u + at8 * 8u : NONE, 0, 0);
                    __builtin_amdgcn_raw_buffer_store_b8(uint8_t(byte), br, have && q == 0 ? at : NONE, 0, 0);
                }
                stores = 2 * FEW;
                if (have && colw + 32 >= a.N && block + 1 < bpr) {  // blocks behind the last column, up to whole steps of the next product
                    stores = 0;
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        for (unsigned b = block + 1; b < bpr; ++b) {
                            const unsigned at = unsigned(m * 16 + c16) * bpr + b;
                            __builtin_amdgcn_raw_buffer_store_b32(0, hr, at * bytes + unsigned(q) * (bytes / 4), 0, 0);
                            if (!fp4) __builtin_amdgcn_raw_buffer_store_b32(0, hr, at * bytes + unsigned(q) * 8u + 4u, 0, 0);
                            __builtin_amdgcn_raw_buffer_store_b8(uint8_t(0), br, q == 0 ? at : NONE, 0, 0);
                        }
                }
            } else if (!regular) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int row = m * 16 + c16;
#pragma unroll
                    for (int n = 0; n < (PAIR ? 2 : 4); ++n) {
                        const int col = colw + n * 16 + 4 * q;
                        const v4f y = value(n, m);
                        if (row < cur.z && col < a.N) mx_store(a, size_t(cur.y + row) * a.ldy + col, min(4, a.N - col), y);
                    }
                }
            } else {
                // stores of 16 bytes that exist whole or not at all: one each, dropped by the descriptor where they do not
                const __amdgpu_buffer_rsrc_t yr = mx_buffer(static_cast<const uint8_t*>(a.Y) + size_t(cur.y) * a.ldy * es,
                                                            size_t(cur.z - 1) * pitch + size_t(a.N) * es);
                if (f32) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int n = 0; n < (PAIR ? 2 : 4); ++n) {
                            const int col = colw + n * 16 + 4 * q;
                            const unsigned off = col < a.N ? unsigned(m * 16 + c16) * pitch + unsigned(col) * 4u : NONE;
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, value(n, m)), yr, off, 0, 0);
                        }
                } else {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int n = 0; n < (PAIR ? 2 : 4); n += 2) {
                            const v4f y0 = value(n, m), y1 = value(n + 1, m);
                            const bool h = a.out == W4A8_F16;
                            uint32_t a0 = h ? f32_to_f16_pair(y0[0], y0[1]) : f32_to_bf16_pair(y0[0], y0[1]);
                            uint32_t a1 = h ? f32_to_f16_pair(y0[2], y0[3]) : f32_to_bf16_pair(y0[2], y0[3]);
                            uint32_t b0 = h ? f32_to_f16_pair(y1[0], y1[1]) : f32_to_bf16_pair(y1[0], y1[1]);
                            uint32_t b1 = h ? f32_to_f16_pair(y1[2], y1[3]) : f32_to_bf16_pair(y1[2], y1[3]);
                            mx_swap16(a0, b0);                  // 8 neighbouring columns: tile n + q % 2, half q / 2
                            mx_swap16(a1, b1);
                            const int col = colw + (n + (q & 1)) * 16 + (q >> 1) * 8;
                            const unsigned off = col < a.N ? unsigned(m * 16 + c16) * pitch + unsigned(col) * 2u : NONE;
                            __builtin_amdgcn_raw_buffer_store_b128(v4i{int(a0), int(a1), int(b0), int(b1)}, yr, off, 0, 0);
                        }
                }
            }
            if (k == mine) break;
        }
    }
}

template <int FMT, bool PAIR, int WN, int MT, bool DEEP>
static void launch_tile_t(const MxArgs& a, int per_cu, hipStream_t s) {
    constexpr long long BM = 16 * MT, cols = PAIR ? 32 * WN : 64 * WN;
    const long long tiles = (a.rows / BM + std::min<long long>(a.E, a.rows)) * ((a.N + cols - 1) / cols);   // an upper bound
    mx_tile_kernel<FMT, PAIR, WN, MT, DEEP><<<dim3(unsigned(std::min<long long>(256 * per_cu, tiles))), dim3(64 * WN), 0, s>>>(a);
}

template <int FMT, bool PAIR>
static void launch_tile_v(const MxArgs& a, MxTile v, hipStream_t s) {
    if (v == MX_TILE_WIDE) launch_tile_t<FMT, PAIR, 8, 8, false>(a, 1, s);
    else if (v == MX_TILE_128) launch_tile_t<FMT, PAIR, 4, 8, false>(a, 2, s);
    else if (v == MX_TILE_64) launch_tile_t<FMT, PAIR, 4, 4, true>(a, 2, s);
    else if (v == MX_TILE_32) launch_tile_t<FMT, PAIR, 4, 2, false>(a, 4, s);
    else launch_tile_t<FMT, PAIR, 2, 2, true>(a, 4, s);
}

void launch_mx_tile(const MxArgs& a, int fmt, bool pair, MxTile v, hipStream_t s) {
    if (fmt == W4A8_MX_FP4) pair ? launch_tile_v<W4A8_MX_FP4, true>(a, v, s) : launch_tile_v<W4A8_MX_FP4, false>(a, v, s);
    else pair ? launch_tile_v<W4A8_MX_FP8, true>(a, v, s) : launch_tile_v<W4A8_MX_FP8, false>(a, v, s);
}

}  // namespace w4a8
