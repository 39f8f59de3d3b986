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

// v, without what the compiler knows of it.  The persistent loop's set-up and epilogue start from it, so that what they
// derive from the lane is computed there and not kept in registers across the MFMA loop, which needs them all.
__device__ __forceinline__ int opaque(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// A tile: rows rbeg .. rbeg + nrows of expert e, column block cb.  Uniform over the workgroup.
struct GroupedTile {
    int e, rbeg, nrows, cb;
};

template <int FMT, bool PAIR>
__global__ __launch_bounds__(512, 2) void moe_grouped_tile_kernel(GroupedArgs a) {
    using acc_t = typename GroupedAcc<FMT>::type;
    constexpr int COLS = PAIR ? GT_N / 2 : GT_N;                // columns of Y
    __shared__ __align__(1024) uint8_t stage0[GT_STAGE];
    __shared__ __align__(1024) uint8_t stage1[GT_STAGE];
    __shared__ int first[GT_MAX_E + 1];                         // row tiles before expert e
    __shared__ float rowscale[2][GT_M];                         // of this tile's rows and the next one's
    __shared__ int wsum[8];
    const lds_ptr st0 = (lds_ptr)stage0, st1 = (lds_ptr)stage1;
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
    // Where K ends inside the last step the chunks behind it receive other bytes of the tile's rows, or what a read past
    // the end of a descriptor gives: they are set to zero in LDS once that step's copies have landed, in both operands,
    // so that an infinity or a NaN there meets nothing.
    const bool ragged = FMT != GF_I8 && (a.kb & 127) != 0;
    auto clear_tail = [&](lds_ptr st) __attribute__((always_inline)) {
        const int row = opaque(int(threadIdx.x));
#pragma unroll 1
        for (int c = (a.kb & 127) >> 4; c < 8; ++c) *(LDS v4i*)(st + row * 128 + (c ^ row_swizzle(row)) * 16) = v4i{0, 0, 0, 0};
        lds_barrier();
    };
    const bool wide = grouped_wide(a);
    // blocks go to the 8 XCDs in turn: the blocks of one XCD take neighbouring tiles, which share rows or columns in its L2
    const int nblk = int(gridDim.x), per = nblk / 8;
    const int rank = nblk % 8 ? int(blockIdx.x) : (int(blockIdx.x) % 8) * per + int(blockIdx.x) / 8;

    auto find = [&](const long long t) __attribute__((always_inline)) {
        const int trow = int(t / ncb);
        int e = 0;                                              // experts that end at or before row tile trow
        for (int c = 0; c < a.E; c += 64)
            e += __popcll(__ballot(c + lane < a.E && first[min(c + lane, a.E - 1) + 1] <= trow));
        e = __builtin_amdgcn_readfirstlane(e);
        const int f0 = __builtin_amdgcn_readfirstlane(first[e]), rt = __builtin_amdgcn_readfirstlane(first[e + 1]) - f0;
        const int in_e = int(t - (long long)f0 * ncb);
        const int panel = in_e / (GT_PANEL * ncb), j = in_e - panel * GT_PANEL * ncb;
        const int rp = min(GT_PANEL, rt - panel * GT_PANEL);
        const int cb = j / rp, rtile = panel * GT_PANEL + j - cb * rp;
        const int r0 = min(max(a.offsets[e], 0), a.rows) + rtile * GT_M;
        return GroupedTile{e, r0, min(GT_M, min(a.offsets[e + 1], a.rows) - r0), cb};
    };

    // Sources of this thread's copies: 4 of the 32 groups of 8 activation rows and 4 of the weights' 32 KiB, as byte
    // offsets from bases that are uniform over the workgroup; each descriptor ends where the tile's data does.
    unsigned xoff[4], woff[4];
    constexpr unsigned WSTEP = FMT == GF_I8 ? 2048 : 128;       // bytes from one step to the next
    __amdgpu_buffer_rsrc_t xr, wr[PAIR ? 2 : 1];                // paired form: gate rows, up rows
    auto fill = [&](lds_ptr st, const int s) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            copy_to_lds(xr, xoff[i], unsigned(s) * 128u, st + (i * 8 + wave) * 1024);
            copy_to_lds(wr[PAIR ? i >> 1 : 0], woff[i], unsigned(s) * WSTEP, st + GT_M * 128 + (i * 8 + wave) * 1024);
        }
    };
    // descriptors, offsets and row scales of a tile, and the copies of its first two steps
    auto begin = [&](const GroupedTile& g, const int buf) __attribute__((always_inline)) {
        const int tid = opaque(int(threadIdx.x)), lane = tid & 63;
        const uint8_t* wexp = a.W + size_t(g.e) * a.expert_stride;
        const int last_col = min(COLS, a.N - g.cb * COLS) - 1;
        xr = a.gather ? buffer_of(a.X, size_t(a.src_rows - 1) * size_t(a.ldx) + size_t(a.kb))
                      : buffer_of(a.X + size_t(g.rbeg) * size_t(a.ldx), size_t(g.nrows - 1) * size_t(a.ldx) + size_t(a.kb));
        if constexpr (FMT == GF_I8) {
            wr[0] = buffer_of(wexp + a.codes_off + size_t(g.cb) * 16 * size_t(steps) * 2048,
                              size_t(last_col / 16 + 1) * size_t(steps) * 2048);
        } else {
#pragma unroll
            for (int p = 0; p < (PAIR ? 2 : 1); ++p)
                wr[p] = buffer_of(wexp + (size_t(g.cb) * COLS + size_t(p) * size_t(a.N)) * a.ldw,
                                  size_t(last_col) * a.ldw + size_t(a.kb));
        }
        int src[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = (i * 8 + wave) * 8 + (lane >> 3);
            const int local = row < g.nrows ? row : 0;
            src[i] = a.gather ? max(grouped_src(a, g.rbeg + local), 0) : local;
        }
        // scale of the tile's row tid; 16 bit: 0 marks a gather entry that names no row
        float rs = 1.0f;
        if (tid < g.nrows && (FMT == GF_I8 || a.gather)) {
            const int r = grouped_src(a, g.rbeg + tid);
            rs = r < 0 ? 0.0f : FMT == GF_I8 ? a.sx[r] : 1.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = (i * 8 + wave) * 8 + (lane >> 3);
            const int chunk = (lane & 7) ^ row_swizzle(row);
            // (opaque products: a fused multiply-add would leave a 64-bit result, two registers for each offset)
            xoff[i] = unsigned(opaque(int(unsigned(src[i]) * unsigned(a.ldx)))) + unsigned(chunk) * 16u;
            if constexpr (FMT == GF_I8) {                       // half a superblock
                const int unit = ((i * 8 + wave) & 1) * 64 + (lane ^ ((lane >> 4) & 1));
                woff[i] = unsigned(min((i * 8 + wave) >> 1, last_col / 16)) * unsigned(steps) * 2048u + unsigned(unit) * 16u;
            } else {
                woff[i] = unsigned(opaque(int(unsigned(min(PAIR ? row & 127 : row, last_col)) * a.ldw))) + unsigned(chunk) * 16u;
            }
        }
        fill(st0, 0);
        if (steps > 1) fill(st1, 1);
        if (tid < GT_M) rowscale[buf][tid] = rs;
    };

    // Operands of half h (64 bytes of K) of a stage: the 4 weight tiles, and 4 of the 8 row tiles.  The compiler may not
    // see into the byte offsets: it would rebuild each address from its terms and lose which stage it belongs to.
    const int wm = wave >> 2, wn = wave & 3;
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

    if (rank >= total) return;
    GroupedTile g = find(rank);
    begin(g, 0);
    int buf = 0;
    for (long long t = rank;; buf ^= 1) {
        acc_t acc[4][8];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int m = 0; m < 8; ++m) acc[n][m] = acc_t{};
        auto mfma = [&](const v4i (&w)[4], const v4i (&x)[4], const int mh) __attribute__((always_inline)) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < 4; ++n) acc[n][mh * 4 + m] = grouped_mfma<FMT>(w[n], x[m], acc[n][mh * 4 + m]);
            __builtin_amdgcn_sched_barrier(0);
        };
        const bool busy = wm * 128 < g.nrows;
        stage_barrier();
        if (ragged && steps == 1) clear_tail(st0);
        if (busy) {
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
                if (ragged && s + 2 == steps) clear_tail(next);
                read_w(next, 0, w0);
                read_x(next, 0, 0, xa);
                if (s + 2 < steps) fill(cur, s + 2);
                mfma(w1, xb, 1);
            };
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
            read_x(last, 0, 1, xb);
            mfma(w0, xa, 0);
            read_w(last, 1, w1);
            read_x(last, 1, 0, xa);
            mfma(w0, xb, 1);
            read_x(last, 1, 1, xb);
            mfma(w1, xa, 0);
            mfma(w1, xb, 1);
        } else {                                                // a wave below the last row only copies
            for (int s = 0; s + 1 < steps; ++s) {
                stage_barrier();
                if (ragged && s + 2 == steps) clear_tail(s & 1 ? st0 : st1);
                if (s + 2 < steps) {
                    if (s & 1) fill(st1, s + 2);
                    else fill(st0, s + 2);
                }
            }
        }
        stage_barrier();

        // the next tile's copies start before this one's outputs are stored
        const GroupedTile cur = g;
        t += nblk;
        const bool more = t < total;
        if (more) {
            g = find(t);
            begin(g, buf ^ 1);
        }
        if (busy) {
            const uint8_t* wexp = a.W + size_t(cur.e) * a.expert_stride;
            const int l = opaque(lane), c16 = l & 15;
            const int col0 = cur.cb * COLS + (PAIR ? wn * 32 : wn * 64) + 4 * (l >> 4);   // this lane in tile n: + 16 n
            constexpr int NT = PAIR ? 2 : 4;
            float4 sw[NT];
            if constexpr (FMT == GF_I8) {
#pragma unroll
                for (int n = 0; n < NT; ++n)                    // padded to whole column tiles: any col < N is inside
                    sw[n] = *reinterpret_cast<const float4*>(wexp + a.scales_off + size_t(min(col0 + n * 16, (a.N - 1) & ~3)) * 4);
            }
            const bool whole = wide && (cur.cb + 1) * COLS <= a.N;      // no column checks
            auto emit = [&](auto store) __attribute__((always_inline)) {
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    const int row = wm * 128 + m * 16 + c16;
                    if (row >= cur.nrows) continue;
                    const float rs = rowscale[buf][row];
                    const size_t at = size_t(cur.rbeg + row) * a.ldy + col0;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float y[4];
                        if constexpr (FMT == GF_I8) {
                            y[0] = (float(acc[n][m][0]) * sw[n].x) * rs;
                            y[1] = (float(acc[n][m][1]) * sw[n].y) * rs;
                            y[2] = (float(acc[n][m][2]) * sw[n].z) * rs;
                            y[3] = (float(acc[n][m][3]) * sw[n].w) * rs;
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float v = PAIR ? silu_mul(acc[n][m][i], acc[n + (PAIR ? 2 : 0)][m][i]) : acc[n][m][i];
                                y[i] = rs == 0.0f ? 0.0f : v;
                            }
                        }
                        store(at + n * 16, col0 + n * 16, y);
                    }
                }
            };
            if (!whole) {
                emit([&](size_t at, int col, const float* y) __attribute__((always_inline)) {
                    if (col < a.N) grouped_store(a, at, min(4, a.N - col), wide, y[0], y[1], y[2], y[3]);
                });
            } else if (!PAIR && a.out == W4A8_F32) {
                emit([&](size_t at, int, const float* y) __attribute__((always_inline)) {
                    *reinterpret_cast<float4*>(static_cast<float*>(a.Y) + at) = make_float4(y[0], y[1], y[2], y[3]);
                });
            } else {
                emit([&](size_t at, int, const float* y) __attribute__((always_inline)) {
                    const uint2 h = FMT == GF_F16 ? make_uint2(f32_to_f16_pair(y[0], y[1]), f32_to_f16_pair(y[2], y[3]))
                                                  : make_uint2(f32_to_bf16_pair(y[0], y[1]), f32_to_bf16_pair(y[2], y[3]));
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.Y) + at) = h;
                });
            }
        }
        if (!more) break;
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
