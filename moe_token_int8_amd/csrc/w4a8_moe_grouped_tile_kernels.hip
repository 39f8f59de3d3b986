// Expert-grouped GEMMs in 8 and 16 bits: the kernel for experts with many rows (MFMA tiles of 256 x 256 and 128 x 128).
//
// Source: P1 "Kimi 2.7 MoE: from 4-bit storage to INT8 (W4A8)" (pwwt.cn), section 4.4 step 4 (the grouped expert GEMM over
// router-sorted rows, "the performance key") and section 5.1 (tiles matched to the MFMA operands).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "w4a8_internal.h"
#include "w4a8_moe_grouped.h"

namespace w4a8 {

// Persistent workgroups of NW waves walk over tiles of 32 NW rows x 32 NW columns (paired form: half of them gate, the
// matching half up columns): one of 8 waves with 256 x 256 tiles on a compute unit, or two of 4 waves with 128 x 128 tiles,
// which read twice the bytes for a product but leave fewer rows and compute units empty.  A step is 128 bytes of K, a cache
// line of every row: the activation rows and as many weight rows are copied straight from memory to LDS (16 bytes a lane,
// no registers in between), into two stages of 64 or 32 KiB, one step ahead of the MFMAs.  (Four stages of 64 bytes keep
// more copies in flight, but ask for every line twice: steps of K = 4096 took 2.0 us against 1.75.)  Wave (wm, wn) owns half
// the rows and 64 columns: NW x 4 MFMA tiles, 128 or 64 accumulators a lane.
constexpr int GT_STEP = 128;                                    // bytes of K in a step
constexpr int GT_PANEL = 4;                                     // row tiles of a panel of consecutive tiles
constexpr int GT_MAX_E = 1024;

// LDS image of a stage: rows of 128 bytes in eight 16-byte chunks, the activations', then the weights'.  Chunk c of row
// r sits at position c ^ row_swizzle(r): 16 rows read at one chunk, and the halves of two neighbouring chunks that the
// LDS serves together, then lie in distinct banks.  Weights in 8-bit codes keep the packed layout's order within 16
// columns, 2 KiB, with neighbouring chunks swapped in the upper 8 columns for the same reason.
__device__ __forceinline__ int row_swizzle(int r) { return (r >> 1) & 7; }

// Stages are addressed as LDS objects, not through generic pointers, and copied into through buffer descriptors: the
// compiler then sees that a read of one stage does not touch the others, and waits neither for the copies in flight into
// them nor (as it does after a global_load_lds) for every LDS read before an MFMA.
#define LDS __attribute__((address_space(3)))
using lds_ptr = LDS uint8_t*;

// (The whole offset is in the register operand: a scalar offset is not part of the descriptor's range check.)
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t src, unsigned off, lds_ptr dst) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (LDS void*)dst, 16, off, 0, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t* base, size_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, int(unsigned(bytes < 0xffffffffu ? bytes : 0xffffffffu)),
                                             0x00020000);
}

// Waits until at most NEWER memory operations of this wave are in flight (the counter goes down in the order of issue)
// and its LDS reads are done, then for every wave.
template <int NEWER>
__device__ __forceinline__ void stage_barrier() {
    static_assert(NEWER < 64, "the counter has 6 bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((NEWER & 15) | ((NEWER >> 4) << 14) | (7 << 4) | (0 << 8));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// v, without what the compiler knows of it.  The persistent loop's set-up and epilogue start from it, so that what they
// derive from the lane is computed there and not kept in registers across the MFMA loop, which needs them all.
__device__ __forceinline__ int opaque(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// Weight column, within a wave's block of 64 (paired form: 32), that MFMA tile n has in its row c.  A lane's sums are the
// rows 4 (lane / 16) .. + 3 of its tiles: with 16-bit outputs the columns are dealt out so that two tiles together give
// it 8 neighbouring ones, a 16-byte store and 64 contiguous bytes a row (8-byte stores in 32-byte pieces cost the
// 8192-token down product 0.04 of 0.68 ms); with float32 a tile's 16 columns are 64 bytes as they stand.
__device__ __forceinline__ int tile_column(bool f32, int n, int c) {
    return f32 ? n * 16 + c : (n >> 1) * 32 + (c >> 2) * 8 + (n & 1) * 4 + (c & 3);
}

template <int FMT, bool PAIR, int NW>
__global__ __launch_bounds__(64 * NW, 2) void moe_grouped_tile_kernel(GroupedArgs a) {
    using acc_t = typename GroupedAcc<FMT>::type;
    constexpr int TILE = 32 * NW, THREADS = 64 * NW;
    constexpr int GT_M = TILE, GT_STAGE = 2 * TILE * GT_STEP;
    constexpr int GT_WOFF = TILE * GT_STEP;                     // weights within a stage
    constexpr int GT_LIST = THREADS;                            // tiles looked up at a time, one a thread
    constexpr int COLS = PAIR ? TILE / 2 : TILE;                // columns of Y
    constexpr int MT = NW;                                      // 16-row tiles of a wave
    __shared__ __align__(1024) uint8_t stage0[GT_STAGE];
    __shared__ __align__(1024) uint8_t stage1[GT_STAGE];
    __shared__ int4 list[GT_LIST];                              // tiles of this workgroup: expert, first row, rows, column block
    __shared__ int first[GT_MAX_E + 1];                         // row tiles before expert e
    __shared__ float rowscale[2][GT_M];                         // of this tile's rows and the next one's
    __shared__ int entries[GT_M];                               // gather entries of the next tile's rows
    __shared__ int wsum[NW];
    const lds_ptr st0 = (lds_ptr)stage0, st1 = (lds_ptr)stage1;
    const int lane = int(threadIdx.x) & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int q = lane >> 4, c16 = lane & 15;
    const int ncb = (a.N + COLS - 1) / COLS;
    const int steps = (a.kb + GT_STEP - 1) / GT_STEP;
    const bool f32 = !PAIR && a.out == W4A8_F32;

    // row tiles of every expert of this launch, as a prefix sum
    {
        constexpr int EPT = GT_MAX_E / THREADS;                 // experts of a thread
        const int tid = threadIdx.x;
        int t[EPT], incl = 0;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const int e = EPT * tid + i;
            // both ends clamped to the rows of the call: whatever the offsets hold, the difference does not overflow
            const int cnt = e < a.E ? min(max(a.offsets[e + 1], 0), a.rows) - min(max(a.offsets[e], 0), a.rows) : 0;
            t[i] = cnt >= a.lo && cnt < a.hi ? (cnt + TILE - 1) / TILE : 0;
            incl += t[i];
        }
        int excl = -incl;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int y = __shfl_up(incl, o, 64);
            if (lane >= o) incl += y;
        }
        if (lane == 63) wsum[wave] = incl;
        __syncthreads();
        for (int w = 0; w < wave; ++w) incl += wsum[w];
        excl += incl;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            if (EPT * tid + i <= a.E) first[EPT * tid + i] = excl;
            excl += t[i];
        }
        if (a.E == GT_MAX_E && tid == THREADS - 1) first[GT_MAX_E] = incl;
        __syncthreads();
    }
    const long long total = (long long)first[a.E] * ncb;
    // blocks go to the 8 XCDs in turn: the blocks of one XCD take neighbouring tiles, which share rows or columns in its L2
    const int nblk = int(gridDim.x), per = nblk / 8;
    const int rank = nblk % 8 ? int(blockIdx.x) : (int(blockIdx.x) % 8) * per + int(blockIdx.x) / 8;
    const int mine = rank < total ? int((total - rank + nblk - 1) / nblk) : 0;      // tiles of this workgroup
    if (mine == 0) return;

    // the tiles from k0 on of this workgroup; all threads, between barriers
    auto look_up = [&](const int k0) __attribute__((always_inline)) {
        const int tid = opaque(int(threadIdx.x));
        if (k0 + tid < mine) {
            const long long t = rank + (long long)(k0 + tid) * nblk;
            const int trow = int(t / ncb);
            int lo = 0, hi = a.E;                               // expert: the last one whose first tile is not after trow
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= trow) lo = mid;
                else hi = mid;
            }
            const int f0 = first[lo], rt = first[lo + 1] - f0, in_e = int(t - (long long)f0 * ncb);
            const int panel = in_e / (GT_PANEL * ncb), j = in_e - panel * GT_PANEL * ncb;
            const int rp = min(GT_PANEL, rt - panel * GT_PANEL);
            const int cb = j / rp, r0 = min(max(a.offsets[lo], 0), a.rows) + (panel * GT_PANEL + j - cb * rp) * GT_M;
            list[tid] = make_int4(lo, r0, min(GT_M, min(a.offsets[lo + 1], a.rows) - r0), cb);
        }
        __syncthreads();
    };

    // Sources of this thread's copies, 4 of the 4 NW groups of 8 activation rows and as many of the weights, as byte offsets
    // from bases that are uniform over the workgroup; each descriptor ends where the tile's data does.  Rows past the
    // tile's last, weight rows past the last column and bytes past the last row's K lie outside it and load nothing.
    unsigned xoff[4], woff;
    __amdgpu_buffer_rsrc_t xr, wr[PAIR ? 2 : 1];                // paired form: gate rows, up rows
    const unsigned tile_bytes = unsigned(steps) * 2048u;        // GF_I8: 16 columns of codes
    const unsigned wgroup = FMT == GF_I8 ? NW / 2 * tile_bytes : 8u * NW * a.ldw;   // from one copy to the next
    // Workgroups that share rows or columns take the steps of every four in another order, each starting at its own: of the
    // lines that they all need, each then fetches a part ahead of the others, and a DRAM page is asked for four
    // neighbouring lines at a time.
    int turn = 0;
    const int whole = a.kb / GT_STEP, whole_fours = whole & ~3;
    const unsigned own_chunk = unsigned(((lane & 7) ^ row_swizzle(wave * 8 + (lane >> 3))) * 16);   // of a row's 128 bytes, in every copy
    auto fill_part = [&](lds_ptr st, const int s0, const int part) __attribute__((always_inline)) {
        const int s = s0 < whole_fours ? (s0 & ~3) | ((s0 + turn) & 3) : s0, i = part >> 1;
        const unsigned wstep = unsigned(s) * (FMT == GF_I8 ? 2048u : GT_STEP);
        // chunks behind K: out of every range, which leaves zeros in LDS, in both operands, so that an infinity or a NaN there
        // meets nothing
        const bool in = s0 < whole || (FMT != GF_I8 && unsigned(s) * GT_STEP + own_chunk < unsigned(a.kb));
        if (part & 1) {
            const unsigned off = woff + (wstep + (PAIR ? i & 1 : i) * wgroup);
            copy_to_lds(wr[PAIR ? i >> 1 : 0], in ? off : 0xfffffff0u, st + GT_WOFF + (i * NW + wave) * 1024);
        } else {
            const unsigned off = xoff[i] + unsigned(s) * GT_STEP;
            copy_to_lds(xr, in ? off : 0xfffffff0u, st + (i * NW + wave) * 1024);
        }
    };
    constexpr int FILL = 8;                                     // copies of a wave in one fill

    // The MFMA loop is two steps long and has no other exit, so that the accumulators stay where they are: an odd number
    // of steps is rounded up with one of zeros.
    const int turns = (steps + 1) / 2;
    auto fill = [&](lds_ptr st, const int s) __attribute__((always_inline)) {
#pragma unroll
        for (int part = 0; part < FILL; ++part) fill_part(st, s, part);
    };
    // Gather entries of a tile's rows, copied to LDS a tile ahead.
    auto request_rows = [&](const int4 g) __attribute__((always_inline)) {
        if (a.gather && wave < GT_M / 64)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(reinterpret_cast<const uint8_t*>(a.gather + g.y), size_t(g.z) * 4),
                                                     (LDS void*)((LDS int*)entries + wave * 64), 4,
                                                     unsigned(opaque(int(threadIdx.x))) * 4u, 0, 0, 0);
    };
    auto source = [&](const int g) __attribute__((always_inline)) {    // row of X, or -1
        if (!a.gather) return g;
        const int t = g < 0 ? -1 : int(unsigned(g) / unsigned(a.topk));
        return t < a.src_rows ? t : -1;
    };
    // scale of row threadIdx.x (16 bit: 1); NO_ROW marks a gather entry that names no row, whose outputs are zeros.  A row whose
    // scale is -0 is taken for one, which has zeros too.
    constexpr float NO_ROW = FMT == GF_I8 ? -0.0f : 0.0f;
    float own_scale = 0.0f;
    // descriptors, offsets and row scales of a tile, and the copies of its first steps
    auto begin = [&](const int4 g) __attribute__((always_inline)) {
        const int tid = opaque(int(threadIdx.x)), lane = tid & 63, wave = tid >> 6;
        const uint8_t* wexp = a.W + size_t(g.x) * a.expert_stride;
        const int last_col = min(COLS, a.N - g.w * COLS) - 1;
        xr = a.gather ? buffer_of(a.X, size_t(a.src_rows - 1) * size_t(a.ldx) + size_t(a.kb))
                      : buffer_of(a.X + size_t(g.y) * size_t(a.ldx), size_t(g.z - 1) * size_t(a.ldx) + size_t(a.kb));
        if constexpr (FMT == GF_I8) {
            wr[0] = buffer_of(wexp + a.codes_off + size_t(g.w) * (COLS / 16) * tile_bytes, size_t(last_col / 16 + 1) * tile_bytes);
        } else {
#pragma unroll
            for (int p = 0; p < (PAIR ? 2 : 1); ++p)
                wr[p] = buffer_of(wexp + (size_t(g.w) * COLS + size_t(p) * size_t(a.N)) * a.ldw,
                                  size_t(last_col) * a.ldw + size_t(a.kb));
        }
        const int own = tid < g.z ? source(a.gather ? entries[tid] : g.y + tid) : -1;
        own_scale = own < 0 ? NO_ROW : 1.0f;
        if (FMT == GF_I8 && own >= 0) own_scale = a.sx[own];
        turn = __builtin_amdgcn_readfirstlane(g.y / GT_M + g.w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {                           // (opaque: a fused multiply-add would leave 64-bit results)
            const int row = (i * NW + wave) * 8 + (lane >> 3), chunk = (lane & 7) ^ row_swizzle(row);
            xoff[i] = unsigned(opaque(int(unsigned(max(source(a.gather ? entries[row] : row), 0)) * unsigned(a.ldx)))) + unsigned(chunk) * 16u;
            if (row >= g.z) xoff[i] = 0xf0000000u;
        }
        if constexpr (FMT == GF_I8) {                           // tile wave / 2 of column block i, half its chunks
            const int p = (wave & 1) * 64 + (lane ^ ((lane >> 4) & 1)), col = tile_column(f32, wave >> 1, (p >> 1) & 15);
            woff = unsigned(opaque(int(unsigned(col >> 4) * tile_bytes))) + unsigned((p >> 5) * 16 + (col & 15)) * 32u +
                   unsigned(p & 1) * 16u;
        } else {
            const int row = wave * 8 + (lane >> 3), n = (wave >> 1) & (PAIR ? 1 : 3);
            const int col = (PAIR ? (wave >> 2) * 32 : 0) + tile_column(f32, n, row & 15);
            woff = unsigned(opaque(int(unsigned(col) * a.ldw))) + unsigned((lane & 7) ^ row_swizzle(row)) * 16u;
        }
        fill(st0, 0);
        fill(st1, 1);
    };

    // Operands of half h (64 bytes of K) of a stage: the 4 weight tiles, and half of the row tiles.  Lane group q takes chunk
    // 4 h + q, the packed layout's order.  The compiler may not see into the byte offsets: it would rebuild each address from
    // its terms and lose which stage it belongs to.
    const int wm = wave / (NW / 2), wn = wave % (NW / 2);
    int xat[2], wat[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int pos = ((4 * h + q) ^ row_swizzle(c16)) * 16;
        xat[h] = opaque((wm * (TILE / 2) + c16) * GT_STEP + pos);
        wat[h] = opaque(GT_WOFF + (FMT == GF_I8 ? wn * 8192 + (2 * lane + (h ^ (c16 >> 3))) * 16
                                                : ((PAIR ? wn * 32 : wn * 64) + c16) * GT_STEP + pos));
    }
    auto read_w = [&](const lds_ptr st, const int h, const int n) __attribute__((always_inline)) {
        return *(const LDS v4i*)(st + wat[h] + (PAIR ? (n >> 1) * (TILE / 2) * GT_STEP + (n & 1) * 2048 : n * 2048));
    };
    auto read_x = [&](const lds_ptr st, const int h, const int m) __attribute__((always_inline)) {
        return *(const LDS v4i*)(st + xat[h] + m * 2048);
    };

    // A tile whose columns come in whole 16-byte stores (of any address) ends, in every wave that computed, with at least
    // STORES of them, which the next tile's first barriers leave in flight.
    constexpr int STORES = PAIR ? MT : 2 * MT;
    const bool near_rows = a.ldy < (size_t(1) << 21);           // 32-bit offsets within a tile
    const int quantum = f32 ? 3 : 7;
    bool behind_stores = false;

    look_up(0);
    int4 g = list[0];
    auto uniform = [&](int4 v) __attribute__((always_inline)) {
        return make_int4(__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y),
                         __builtin_amdgcn_readfirstlane(v.z), __builtin_amdgcn_readfirstlane(v.w));
    };
    g = uniform(g);
    request_rows(g);
    stage_barrier<0>();
    begin(g);
    for (int k = 0;;) {
        const int4 cur = g;
        const int buf = k & 1;
        if (behind_stores) stage_barrier<FILL + STORES>();
        else stage_barrier<0>();
        if (threadIdx.x < GT_M) rowscale[buf][threadIdx.x] = own_scale;
        // the next tile, and its gather entries: requested here, first needed at the end of this tile
        if (++k < mine) {
            if (k % GT_LIST == 0) look_up(k);
            g = uniform(list[k % GT_LIST]);
            request_rows(g);
        }
        if (wm * (TILE / 2) < cur.z) {
            acc_t acc[4][MT];
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[n][m] = acc_t{};
            // 4 of the 8 MT MFMAs of a step: row tile m against the 4 weight tiles
            auto mfma4 = [&](const v4i (&w)[4], const v4i x, const int m) __attribute__((always_inline)) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int n = 0; n < 4; ++n) acc[n][m] = grouped_mfma<FMT>(w[n], x, acc[n][m]);
                __builtin_amdgcn_sched_barrier(0);
            };
            constexpr int H = MT / 2, WR = 4 / H, CP = FILL / H;   // row tiles, weight reads and copies of a group
            v4i wa[4], wb[4], xa[H], xb[H];
            // One step: four groups of 4 H MFMAs, the operands of each read from LDS during the group before it.  The barrier
            // stands before the last group, when this step's last operands are in registers: behind it the next stage is
            // whole and this one is free for the copies of the step after.
            auto step = [&](const lds_ptr st, const lds_ptr next, const int s, const bool early) __attribute__((always_inline)) {
#pragma unroll
                for (int m = 0; m < H; ++m) {
                    xb[m] = read_x(st, 0, H + m);
                    mfma4(wa, xa[m], m);
                }
#pragma unroll
                for (int m = 0; m < H; ++m) {
#pragma unroll
                    for (int n = m * WR; n < (m + 1) * WR; ++n) wb[n] = read_w(st, 1, n);
                    xa[m] = read_x(st, 1, m);
                    mfma4(wa, xb[m], H + m);
                }
#pragma unroll
                for (int m = 0; m < H; ++m) {
                    xb[m] = read_x(st, 1, H + m);
                    mfma4(wb, xa[m], m);
                }
                if (early) stage_barrier<STORES>();
                else stage_barrier<0>();
                const bool more = s + 2 < 2 * turns;
#pragma unroll
                for (int m = 0; m < H; ++m) {
#pragma unroll
                    for (int n = m * WR; n < (m + 1) * WR; ++n) wa[n] = read_w(next, 0, n);
                    xa[m] = read_x(next, 0, m);
                    if (more) {
#pragma unroll
                        for (int part = m * CP; part < (m + 1) * CP; ++part) fill_part(st, s + 2, part);
                    }
                    mfma4(wb, xb[m], H + m);
                }
            };
#pragma unroll
            for (int n = 0; n < 4; ++n) wa[n] = read_w(st0, 0, n);
#pragma unroll
            for (int m = 0; m < H; ++m) xa[m] = read_x(st0, 0, m);
            for (int s = 0; s < steps; s += 2) {
                step(st0, st1, s, behind_stores && s == 0);
                step(st1, st0, s + 1, false);
            }

            const int l = opaque(lane), c16 = l & 15;
            constexpr int NT = PAIR ? 2 : 4;
            int col[NT];                                        // of this lane's four sums in tile n
#pragma unroll
            for (int n = 0; n < NT; ++n) col[n] = cur.w * COLS + (PAIR ? wn * 32 : wn * 64) + tile_column(f32, n, 4 * (l >> 4));
            float4 sw[NT];
            if constexpr (FMT == GF_I8) {
                const uint8_t* scales = a.W + size_t(cur.x) * a.expert_stride + a.scales_off;
#pragma unroll
                for (int n = 0; n < NT; ++n)                    // padded to whole column tiles: any col < N is inside
                    sw[n] = *reinterpret_cast<const float4*>(scales + size_t(min(col[n], (a.N - 1) & ~3)) * 4);
            }
            // every stage has been read: the next tile's copies start before this one's outputs are stored
            lds_barrier();
            if (k < mine) begin(g);
            auto value = [&](const int n, const int m, const float rs, float* y) __attribute__((always_inline)) {
                if constexpr (FMT == GF_I8) {
                    y[0] = (float(acc[n][m][0]) * sw[n].x) * rs;
                    y[1] = (float(acc[n][m][1]) * sw[n].y) * rs;
                    y[2] = (float(acc[n][m][2]) * sw[n].z) * rs;
                    y[3] = (float(acc[n][m][3]) * sw[n].w) * rs;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = PAIR ? silu_gate(acc[n][m][i]) * acc[n + (PAIR ? 2 : 0)][m][i] : acc[n][m][i];
                }
            };
            // the outputs of a gather entry that names no row: zeros, whatever its stand-in row and the weights' scales hold
            auto none = [&](const float rs) __attribute__((always_inline)) {
                return FMT == GF_I8 ? __float_as_uint(rs) == __float_as_uint(NO_ROW) : rs == NO_ROW;
            };
            // stores of 16 bytes that exist whole or not at all: one each, dropped by the descriptor where they do not
            const bool regular = near_rows && ((a.N & quantum) == 0 || (cur.w + 1) * COLS <= a.N);
            const unsigned es = f32 ? 4u : 2u, pitch = unsigned(a.ldy) * es;
            const __amdgpu_buffer_rsrc_t yr = buffer_of(static_cast<const uint8_t*>(a.Y) + size_t(cur.y) * a.ldy * es,
                                                        size_t(cur.z - 1) * pitch + size_t(a.N) * es);
            unsigned coff[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) coff[n] = col[n] < a.N ? unsigned(col[n]) * es : 0x80000000u;
            float rs[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) rs[m] = rowscale[buf][wm * (TILE / 2) + m * 16 + c16];
            if (!regular) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int row = wm * (TILE / 2) + m * 16 + c16;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float y[4];
                        value(n, m, rs[m], y);
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[i] = none(rs[m]) ? 0.0f : y[i];
                        if (row < cur.z && col[n] < a.N)
                            grouped_store(a, size_t(cur.y + row) * a.ldy + col[n], min(4, a.N - col[n]), y[0], y[1], y[2], y[3]);
                    }
                }
            } else if (f32) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const unsigned at = unsigned(wm * (TILE / 2) + m * 16 + c16) * pitch;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float y[4];
                        value(n, m, rs[m], y);
                        const v4i h = __builtin_bit_cast(v4i, v4f{y[0], y[1], y[2], y[3]});
                        __builtin_amdgcn_raw_buffer_store_b128(none(rs[m]) ? v4i{0, 0, 0, 0} : h, yr, at + coff[n], 0, 0);
                    }
                }
            } else {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const unsigned at = unsigned(wm * (TILE / 2) + m * 16 + c16) * pitch;
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        float y[2][4];
                        value(n, m, rs[m], y[0]);
                        value(n + 1, m, rs[m], y[1]);
                        v4i h;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float lo = y[i >> 1][2 * (i & 1)], hi = y[i >> 1][2 * (i & 1) + 1];
                            h[i] = int(FMT == GF_F16 ? f32_to_f16_pair(lo, hi) : f32_to_bf16_pair(lo, hi));
                        }
                        __builtin_amdgcn_raw_buffer_store_b128(none(rs[m]) ? v4i{0, 0, 0, 0} : h, yr, at + coff[n], 0, 0);
                    }
                }
            }
            if (k == mine) break;
            behind_stores = regular && steps >= 2;
        } else {                                                // a wave below the last row only copies
            for (int s = 0; s < 2 * turns; ++s) {
                if (s == 0 && behind_stores) stage_barrier<STORES>();
                else stage_barrier<0>();
                if (s + 2 < 2 * turns) fill(s & 1 ? st1 : st0, s + 2);
            }
            lds_barrier();
            if (k == mine) break;
            begin(g);
            behind_stores = false;                              // no stores behind its copies
        }
    }
}

// Which tiles a call takes, and about how long they take, in us.  The host knows rows and E: an expert with more than 64
// rows ends in a tile that is filled by half on average, and such experts are no more than rows / (65 + rows / E).  A round
// of 256 large tiles takes 9.7 us and 1.6 us for 128 bytes of K, a round of 512 small ones 8 and 1.0 (with one workgroup a
// compute unit 0.85, in 8 bits 0.55).  Measured, small / large: 8192 tokens x 6 of 64 experts, K = 1408, N = 4096: 683 /
// 588 us; in 8 bits, K = 4096, N = 2816: 672 / 570; 4837 x 8 of 220, K = 768, N = 512: 88 / 80; 556 x 8 of 111, K = 1336,
// I = 1786: 296 / 308; 787 x 5 of 6, K = 3200, N = 632 in 8 bits: 31 / 48; 4346 x 3 of 19, K = 2984, N = 256: 55 / 90.
TileChoice choose_tiles(const GroupedArgs& a, bool i8, bool pair) {
    const double rows = a.rows, steps = (a.kb + GT_STEP - 1) / GT_STEP, width = pair ? 2.0 * a.N : a.N;
    const double ends = 0.5 * std::min(double(a.E), rows / (65 + rows / a.E));
    const double large = (std::floor(rows / 256) + ends) * std::ceil(width / 256);
    const double small = (std::floor(rows / 128) + ends) * std::ceil(width / 128);
    const double us_large = std::ceil(large / 256) * (9.7 + 1.6 * steps);
    const double us_small = std::ceil(small / 512) * (8 + (small > 256 ? 1.0 : i8 ? 0.55 : 0.85) * steps);
    return us_small < us_large ? TileChoice{true, us_small} : TileChoice{false, us_large};
}

template <int FMT, bool PAIR>
static bool launch_tile_t(const GroupedArgs& a, hipStream_t s) {
    auto tiles = [&](long long tile) {                          // an upper bound
        const long long cols = PAIR ? tile / 2 : tile;
        return (a.rows / tile + std::min<long long>(a.E, a.rows / a.lo)) * ((a.N + cols - 1) / cols);
    };
    const bool small = choose_tiles(a, FMT == GF_I8, PAIR).small;
    if (tiles(256) == 0) return small;
    if (small)
        moe_grouped_tile_kernel<FMT, PAIR, 4><<<dim3(unsigned(std::min<long long>(512, tiles(128)))), dim3(256), 0, s>>>(a);
    else
        moe_grouped_tile_kernel<FMT, PAIR, 8><<<dim3(unsigned(std::min<long long>(256, tiles(256)))), dim3(512), 0, s>>>(a);
    return small;
}

bool launch_grouped_tile(const GroupedArgs& a, int fmt, bool pair, hipStream_t s) {
    if (fmt == GF_I8) return launch_tile_t<GF_I8, false>(a, s);
    if (fmt == GF_BF16) return pair ? launch_tile_t<GF_BF16, true>(a, s) : launch_tile_t<GF_BF16, false>(a, s);
    return pair ? launch_tile_t<GF_F16, true>(a, s) : launch_tile_t<GF_F16, false>(a, s);
}

}  // namespace w4a8
