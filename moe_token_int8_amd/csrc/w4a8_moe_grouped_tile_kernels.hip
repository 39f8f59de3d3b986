// Expert-grouped GEMMs in 8 and 16 bits: the kernel for experts with many rows (256 x 256 MFMA tiles).
//
// Source: P1 "Kimi 2.7 MoE: from 4-bit storage to INT8 (W4A8)" (pwwt.cn), section 4.4 step 4 (the grouped expert GEMM over
// router-sorted rows, "the performance key") and section 5.1 (tiles matched to the MFMA operands).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "w4a8_internal.h"
#include "w4a8_moe_grouped.h"

namespace w4a8 {

// A persistent workgroup of 8 waves per compute unit walks over 256-row x 256-column tiles (paired form: 128 gate and the
// matching 128 up columns).  Per step of 128 bytes of K the 256 activation rows and the 256 weight rows are copied
// straight from memory to LDS (global_load_lds, 16 bytes a lane, no registers in between), one step ahead of the MFMAs:
// two 64 KiB stages.  Wave (wm, wn) owns rows 128 wm .. + 127 and 64 columns: 8 x 4 MFMA tiles, 128 accumulators a lane.
constexpr int GT_M = 256, GT_N = 256;
constexpr int GT_STAGE = (GT_M + GT_N) * 128;
constexpr int GT_PANEL = 4;                                     // row tiles of a panel of consecutive tiles
constexpr int GT_MAX_E = 1024;

// LDS image of a stage: the activation rows, then the weight rows, 128 bytes each, in 16-byte chunks.  Chunk c of row r
// sits at position c ^ ((r >> 1) & 7): the 16 rows that an operand read takes at one chunk then lie in distinct banks.  A
// copy of 64 lanes fills 8 rows in order, so lane l supplies row l / 8, position l % 8.  Packed codes keep their
// superblocks of 2 KiB (16 columns) with neighbouring chunks swapped in the upper 8 columns, for the same reason.
__device__ __forceinline__ int row_swizzle(int r) { return (r >> 1) & 7; }

// Chunk that lane group q takes of half h: the packed layout's order, for the 16-bit rows too.  (With the streaming
// kernel's order 2 q + h two lane groups that are served together meet in the same banks.)
__device__ __forceinline__ int operand_chunk(int q, int h) { return 4 * h + q; }

// Stages are addressed as LDS objects, not through generic pointers, and copied into through buffer descriptors: the
// compiler then sees that a read of one stage does not touch the other, and waits neither for the copies in flight into
// it nor (as it does after a global_load_lds) for every LDS read before an MFMA.
#define LDS __attribute__((address_space(3)))
using lds_ptr = LDS uint8_t*;

__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t src, unsigned off, unsigned step, lds_ptr dst) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (LDS void*)dst, 16, off, step, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t* base, size_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, int(unsigned(bytes < 0xffffffffu ? bytes : 0xffffffffu)),
                                             0x00020000);
}

// Every copy of this wave has landed and every wave is here: the stage that was being filled is whole and the one that
// was being read is free.
__device__ __forceinline__ void stage_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((7 << 4) | (0 << 8));           // vmcnt 0, lgkmcnt 0, expcnt not waited for
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int FMT, bool PAIR>
__global__ __launch_bounds__(512, 2) void moe_grouped_tile_kernel(GroupedArgs a) {
    using acc_t = typename GroupedAcc<FMT>::type;
    constexpr int COLS = PAIR ? GT_N / 2 : GT_N;                // columns of Y
    __shared__ __align__(1024) uint8_t stage0[GT_STAGE];
    __shared__ __align__(1024) uint8_t stage1[GT_STAGE];
    __shared__ int first[GT_MAX_E + 1];                         // row tiles before expert e
    __shared__ int wsum[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, c16 = lane & 15;

    // row tiles of every expert of this launch, as a prefix sum (two experts a thread)
    {
        int t[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = 2 * tid + i;
            const int cnt = e < a.E ? min(a.offsets[e + 1], a.rows) - min(max(a.offsets[e], 0), a.rows) : 0;
            t[i] = cnt >= a.lo && cnt < a.hi ? (cnt + GT_M - 1) / GT_M : 0;
        }
        int incl = t[0] + t[1];
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int y = __shfl_up(incl, o, 64);
            if (lane >= o) incl += y;
        }
        if (lane == 63) wsum[wave] = incl;
        __syncthreads();
        for (int w = 0; w < wave; ++w) incl += wsum[w];
        const int excl = incl - t[0] - t[1];
        if (2 * tid <= a.E) first[2 * tid] = excl;
        if (2 * tid + 1 <= a.E) first[2 * tid + 1] = excl + t[0];
        if (a.E == GT_MAX_E && tid == 511) first[GT_MAX_E] = incl;
        __syncthreads();
    }
    const int ncb = (a.N + COLS - 1) / COLS;
    const long long total = (long long)first[a.E] * ncb;
    const int steps = (a.kb + 127) / 128;
    const bool wide = grouped_wide(a);
    // blocks go to the 8 XCDs in turn: the blocks of one XCD take neighbouring tiles, which share rows or columns in its L2
    const int nblk = int(gridDim.x), per = nblk / 8;
    const int rank = nblk % 8 ? int(blockIdx.x) : (int(blockIdx.x) % 8) * per + int(blockIdx.x) / 8;

    for (long long t = rank; t < total; t += nblk) {
        // expert of the tile: the last one whose first tile is not after it
        const int trow = int(t / ncb);
        int lo = 0, hi = a.E;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= trow) lo = mid;
            else hi = mid;
        }
        const int e = __builtin_amdgcn_readfirstlane(lo);
        const int rt = first[e + 1] - first[e];
        const int in_e = int(t - (long long)first[e] * ncb);
        const int panel = in_e / (GT_PANEL * ncb), j = in_e - panel * GT_PANEL * ncb;
        const int rp = min(GT_PANEL, rt - panel * GT_PANEL);
        const int rtile = __builtin_amdgcn_readfirstlane(panel * GT_PANEL + j % rp);
        const int cb = __builtin_amdgcn_readfirstlane(j / rp);
        const int rbeg = __builtin_amdgcn_readfirstlane(min(max(a.offsets[e], 0), a.rows)) + rtile * GT_M;
        const int nrows = min(GT_M, __builtin_amdgcn_readfirstlane(min(a.offsets[e + 1], a.rows)) - rbeg);
        const uint8_t* wexp = a.W + size_t(e) * a.expert_stride;

        // Sources of this thread's copies: 4 of the 32 groups of 8 activation rows and 4 of the weights' 32 KiB, as byte
        // offsets from bases that are uniform over the workgroup; each descriptor ends where the tile's data does.
        unsigned xoff[4], woff[4];
        constexpr unsigned WSTEP = FMT == GF_I8 ? 2048 : 128;   // bytes from one step to the next
        const int last_col = min(COLS, a.N - cb * COLS) - 1;
        const __amdgpu_buffer_rsrc_t xr =
            a.gather ? buffer_of(a.X, size_t(a.src_rows - 1) * size_t(a.ldx) + size_t(a.kb))
                     : buffer_of(a.X + size_t(rbeg) * size_t(a.ldx), size_t(nrows - 1) * size_t(a.ldx) + size_t(a.kb));
        __amdgpu_buffer_rsrc_t wr[PAIR ? 2 : 1];                // paired form: gate rows, up rows
        if constexpr (FMT == GF_I8) {
            wr[0] = buffer_of(wexp + a.codes_off + size_t(cb) * 16 * size_t(steps) * 2048,
                              size_t(last_col / 16 + 1) * size_t(steps) * 2048);
        } else {
#pragma unroll
            for (int p = 0; p < (PAIR ? 2 : 1); ++p)
                wr[p] = buffer_of(wexp + (size_t(cb) * COLS + size_t(p) * size_t(a.N)) * a.ldw, size_t(last_col) * a.ldw + size_t(a.kb));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = (i * 8 + wave) * 8 + (lane >> 3);
            const int chunk = (lane & 7) ^ row_swizzle(row);
            const int local = row < nrows ? row : 0;
            const int src = a.gather ? max(grouped_src(a, rbeg + local), 0) : local;
            xoff[i] = unsigned(src) * unsigned(a.ldx) + unsigned(chunk) * 16u;
            if constexpr (FMT == GF_I8) {                       // half a superblock
                const int unit = ((i * 8 + wave) & 1) * 64 + (lane ^ ((lane >> 4) & 1));
                woff[i] = unsigned(min((i * 8 + wave) >> 1, last_col / 16)) * unsigned(steps) * 2048u + unsigned(unit) * 16u;
            } else {
                woff[i] = unsigned(min(PAIR ? row & 127 : row, last_col)) * a.ldw + unsigned(chunk) * 16u;
            }
        }
        // Where K ends inside the last step the chunks behind it hold other bytes of the tile's rows, or nothing at the
        // end of the descriptor; they are masked when they are read.
        const bool ragged = FMT != GF_I8 && (a.kb & 127) != 0;
        auto fill = [&](lds_ptr st, const int s) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                copy_to_lds(xr, xoff[i], unsigned(s) * 128u, st + (i * 8 + wave) * 1024);
                copy_to_lds(wr[PAIR ? i >> 1 : 0], woff[i], unsigned(s) * WSTEP, st + GT_M * 128 + (i * 8 + wave) * 1024);
            }
        };

        const int wm = wave >> 2, wn = wave & 3;
        acc_t acc[4][8];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int m = 0; m < 8; ++m) acc[n][m] = acc_t{};
        // Operands of half h (64 bytes of K) of a stage: the 4 weight tiles, and 4 of the 8 row tiles.  The compiler may not
        // see into the byte offsets: it would rebuild each address from its terms and lose which stage it belongs to.
        int xat[2], wat[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int pos = (operand_chunk(q, h) ^ row_swizzle(c16)) * 16;
            xat[h] = (wm * 128 + c16) * 128 + pos;
            if constexpr (FMT == GF_I8) wat[h] = GT_M * 128 + wn * 4 * 2048 + (2 * lane + (h ^ (c16 >> 3))) * 16;
            else wat[h] = GT_M * 128 + ((PAIR ? wn * 32 : wn * 64) + c16) * 128 + pos;
            asm volatile("" : "+v"(xat[h]), "+v"(wat[h]));
        }
        auto read_w = [&](const lds_ptr st, const int h, v4i (&w)[4]) __attribute__((always_inline)) {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                w[n] = *(const LDS v4i*)(st + wat[h] + (PAIR ? (n >> 1) * 128 * 128 + (n & 1) * 2048 : n * 2048));
        };
        auto read_x = [&](const lds_ptr st, const int h, const int mh, v4i (&x)[4]) __attribute__((always_inline)) {
#pragma unroll
            for (int m = 0; m < 4; ++m) x[m] = *(const LDS v4i*)(st + xat[h] + (mh * 4 + m) * 2048);
        };
        auto mfma = [&](const v4i (&w)[4], const v4i (&x)[4], const int mh) __attribute__((always_inline)) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < 4; ++n) acc[n][mh * 4 + m] = grouped_mfma<FMT>(w[n], x[m], acc[n][mh * 4 + m]);
            __builtin_amdgcn_sched_barrier(0);
        };
        const lds_ptr st0 = (lds_ptr)stage0, st1 = (lds_ptr)stage1;
        fill(st0, 0);
        if (wm * 128 < nrows) {
            v4i w0[4], w1[4], xa[4], xb[4];
            // One step: four groups of 16 MFMAs, the operands of each read from LDS during the group before it.  The
            // barrier stands before the last group, when this step's last operands are in registers: behind it the next
            // stage is whole and this one is free for the copies of the step after.
            auto step = [&](const lds_ptr cur, const lds_ptr next, const int s) __attribute__((always_inline)) {
                read_x(cur, 0, 1, xb);
                mfma(w0, xa, 0);
                read_w(cur, 1, w1);
                read_x(cur, 1, 0, xa);
                mfma(w0, xb, 1);
                read_x(cur, 1, 1, xb);
                mfma(w1, xa, 0);
                stage_barrier();
                read_w(next, 0, w0);
                read_x(next, 0, 0, xa);
                if (s + 2 < steps) fill(cur, s + 2);
                mfma(w1, xb, 1);
            };
            stage_barrier();
            if (steps > 1) fill(st1, 1);
            read_w(st0, 0, w0);
            read_x(st0, 0, 0, xa);
            int s = 0;
            for (; s + 2 < steps; s += 2) {
                step(st0, st1, s);
                step(st1, st0, s + 1);
            }
            if (s + 1 < steps) step(st0, st1, s++);
            // last step
            const lds_ptr last = s & 1 ? st1 : st0;
            auto masked = [&](const int h, v4i (&w)[4], v4i (&x)[4], const bool new_w) __attribute__((always_inline)) {
                if (!ragged) return;
                const bool in = s * 128 + operand_chunk(q, h) * 16 < a.kb;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = in ? x[i] : v4i{0, 0, 0, 0};
                    if (new_w) w[i] = in ? w[i] : v4i{0, 0, 0, 0};
                }
            };
            read_x(last, 0, 1, xb);
            masked(0, w0, xa, true);
            mfma(w0, xa, 0);
            read_w(last, 1, w1);
            read_x(last, 1, 0, xa);
            masked(0, w0, xb, false);
            mfma(w0, xb, 1);
            read_x(last, 1, 1, xb);
            masked(1, w1, xa, true);
            mfma(w1, xa, 0);
            masked(1, w1, xb, false);
            mfma(w1, xb, 1);
        } else {                                                // a wave below the last row only copies
            stage_barrier();
            if (steps > 1) fill(st1, 1);
            for (int s = 0; s + 1 < steps; ++s) {
                stage_barrier();
                if (s + 2 < steps) fill(s & 1 ? st1 : st0, s + 2);
            }
        }
        const bool busy = wm * 128 < nrows;
        stage_barrier();                                        // the next tile's first copies overwrite stage 0

        if (busy) {
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                const int row = wm * 128 + m * 16 + c16;
                if (row >= nrows) continue;
                const int src = grouped_src(a, rbeg + row);
                const float sxr = FMT == GF_I8 && src >= 0 ? a.sx[src] : 0.0f;
#pragma unroll
                for (int n = 0; n < (PAIR ? 2 : 4); ++n) {
                    const int col = cb * COLS + (PAIR ? wn * 32 : wn * 64) + n * 16 + 4 * q;
                    if (col >= a.N) continue;
                    float y[4];
                    if constexpr (FMT == GF_I8) {
                        const float4 sw4 = *reinterpret_cast<const float4*>(wexp + a.scales_off + size_t(col) * 4);
                        y[0] = (float(acc[n][m][0]) * sw4.x) * sxr;
                        y[1] = (float(acc[n][m][1]) * sw4.y) * sxr;
                        y[2] = (float(acc[n][m][2]) * sw4.z) * sxr;
                        y[3] = (float(acc[n][m][3]) * sw4.w) * sxr;
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float v = PAIR ? silu_mul(acc[n][m][i], acc[n + (PAIR ? 2 : 0)][m][i]) : acc[n][m][i];
                            y[i] = src < 0 ? 0.0f : v;
                        }
                    }
                    grouped_store(a, size_t(rbeg + row) * a.ldy + col, min(4, a.N - col), wide, y[0], y[1], y[2], y[3]);
                }
            }
        }
    }
}

template <int FMT, bool PAIR>
static void launch_tile_t(const GroupedArgs& a, int blocks, hipStream_t s) {
    moe_grouped_tile_kernel<FMT, PAIR><<<dim3(unsigned(blocks)), dim3(512), 0, s>>>(a);
}

void launch_grouped_tile(const GroupedArgs& a, int fmt, bool pair, hipStream_t s) {
    // one workgroup a compute unit, fewer when the call has fewer tiles
    const long long ncb = (a.N + (pair ? GT_N / 2 : GT_N) - 1) / (pair ? GT_N / 2 : GT_N);
    const long long tiles = (a.rows / GT_M + std::min<long long>(a.E, a.rows / a.lo)) * ncb;
    const int blocks = int(std::min<long long>(256, tiles));
    if (blocks == 0) return;
    if (fmt == GF_I8) launch_tile_t<GF_I8, false>(a, blocks, s);
    else if (fmt == GF_BF16 && pair) launch_tile_t<GF_BF16, true>(a, blocks, s);
    else if (fmt == GF_BF16) launch_tile_t<GF_BF16, false>(a, blocks, s);
    else if (pair) launch_tile_t<GF_F16, true>(a, blocks, s);
    else launch_tile_t<GF_F16, false>(a, blocks, s);
}

}  // namespace w4a8
