// Quantisation to the microscaled formats, its inverse, and the packing of MXFP4 weights.
//
// Sources (cited with the page's own section names):
//   P3 "Quantization: formats, error and the real execution path" (wineandchord.com): the microscaled formats beside the
//      integer ones (FP4, FP8 and their block scales).
//   P2 "Kimi 2.7 MoE W4A8: 4-bit storage to INT8, deployment notes" (xdnf.cn), section 3.3: a quantize node before each Linear.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>

#include "w4a8_mx.h"

namespace w4a8 {

// Rows -> codes and scales.  A lane takes 8 neighbours along K (16 or 32 bytes in, 4 or 8 out), 4 lanes a block, a wave 512
// of a row; the block's maximum is two quad permutes.  Bound by the copy: 2 bytes in and 17/32 or 33/32 out an element (8192 x
// 7168 bfloat16 -> fp4: 31 us, 4.8 TB/s).
template <int DT, int FMT>
__device__ __forceinline__ void quant_chunk(const uint8_t* X, const long long M, const int K, const long long ldx, const int chunks,
                                            uint8_t* Xq, uint8_t* sx, const long long w, const int lane) {
    constexpr int ES = DT == W4A8_F32 ? 4 : 2;
    const int Kp = mx_kp(K);
    const long long row = w / chunks;
    const int k = int(w - row * chunks) * 512 + lane * 8;
    if (row >= M || k >= Kp) return;                            // whole blocks of 4 lanes: Kp is a multiple of 128
    float v[8];
    mx_load8<DT>(X + (size_t(row) * size_t(ldx) + size_t(min(k, K))) * ES, K - k, v);
    const uint32_t byte = mx_scale_byte<FMT>(mx_quad_max(mx_amax8(v)));
    const uint2 q = mx_encode8<FMT>(v, byte);
    if constexpr (FMT == W4A8_MX_FP4) *reinterpret_cast<uint32_t*>(Xq + size_t(row) * size_t(Kp / 2) + k / 2) = q.x;
    else *reinterpret_cast<uint2*>(Xq + size_t(row) * size_t(Kp) + k) = q;
    if ((lane & 3) == 0) sx[size_t(row) * size_t(Kp / 32) + k / 32] = uint8_t(byte);
}

template <int DT, int FMT>
__global__ __launch_bounds__(256) void mx_quant_kernel(const uint8_t* X, long long M, int K, long long ldx, int chunks,
                                                       uint8_t* Xq, uint8_t* sx) {
    const long long w = (long long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    quant_chunk<DT, FMT>(X, M, K, ldx, chunks, Xq, sx, w, int(threadIdx.x) & 63);
}

// One expert's part of the order of the routed rows, by one wave: ids below e count towards the expert's first place, ids equal to
// e take the next places in their order, and each wave reads all ids for itself, so that no wave waits for another.  (The same
// results as a counting sort in one workgroup, which is the quicker way for many ids.)
__device__ __forceinline__ void route_expert(const int* ids, const int R, const int E, const int e, int* rows, int* offs, int* inv,
                                             const int lane) {
    int below = 0, mine = 0;
    for (int c = 0; c < R; c += 1024) {                         // 16 loads in flight
        int id[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int r = c + j * 64 + lane;
            id[j] = r < R ? ids[r] : -1;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            below += __popcll(__ballot(id[j] >= 0 && id[j] < e));
            mine += __popcll(__ballot(id[j] == e));
        }
    }
    if (lane == 0) {
        offs[e] = below;
        if (e == E - 1) offs[E] = below + mine;
    }
    if (!mine && e != 0) return;
    for (int c = 0; c < R; c += 1024) {
        int id[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int r = c + j * 64 + lane;
            id[j] = r < R ? ids[r] : E;
            if (e == 0 && r < R && (id[j] < 0 || id[j] >= E)) inv[r] = -1;      // counted nowhere
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const unsigned long long hit = __ballot(id[j] == e);
            const int at = below + __popcll(hit & ((1ull << lane) - 1)), r = c + j * 64 + lane;
            if (id[j] == e) rows[at] = r, inv[r] = at;
            below += __popcll(hit);
        }
    }
}

// The first steps of an expert layer in one launch: the order of the routed rows, by the first workgroups (a wave an expert), and
// the codes of the tokens, by the others.
template <int FMT>
__global__ __launch_bounds__(256) void mx_route_quant_kernel(const int* ids, int R, int E, int* rows, int* offs, int* inv,
                                                             const uint8_t* X, int M, int K, int chunks, uint8_t* Xq, uint8_t* sx) {
    const int lane = int(threadIdx.x) & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int routing = (E + 3) / 4;
    if (int(blockIdx.x) < routing) {
        const int e = int(blockIdx.x) * 4 + wave;
        if (e < E) route_expert(ids, R, E, e, rows, offs, inv, lane);
    } else {
        quant_chunk<W4A8_BF16, FMT>(X, M, K, K, chunks, Xq, sx, (long long)(int(blockIdx.x) - routing) * 4 + wave, lane);
    }
}

// Codes and scales -> values: 8 a lane.
template <int FMT, int DT>
__global__ __launch_bounds__(256) void mx_dequant_kernel(const uint8_t* Xq, const uint8_t* sx, long long M, int K, int chunks,
                                                         uint8_t* Y, long long ldy) {
    constexpr int ES = DT == W4A8_F32 ? 4 : 2;
    const int lane = int(threadIdx.x) & 63, Kp = mx_kp(K);
    const long long w = (long long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const long long row = w / chunks;
    const int k = int(w - row * chunks) * 512 + lane * 8;
    if (row >= M || k >= K) return;
    const float s = mx_scale_value(sx[size_t(row) * size_t(Kp / 32) + k / 32]);
    float v[8];
    if constexpr (FMT == W4A8_MX_FP4) {
        const uint32_t q = *reinterpret_cast<const uint32_t*>(Xq + size_t(row) * size_t(Kp / 2) + k / 2);
        auto two = [&](const v2f t, int i) __attribute__((always_inline)) { v[i] = t[0], v[i + 1] = t[1]; };
        two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0), 0);
        two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1), 2);
        two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2), 4);
        two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3), 6);
    } else {
        const uint2 q = *reinterpret_cast<const uint2*>(Xq + size_t(row) * size_t(Kp) + k);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int d = int(h ? q.y : q.x);
            const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8(d, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(d, true);
            v[4 * h] = a[0], v[4 * h + 1] = a[1], v[4 * h + 2] = b[0], v[4 * h + 3] = b[1];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s;
    mx_store8<DT>(Y + (size_t(row) * size_t(ldy) + size_t(k)) * ES, K - k, v);
}

// Weights -> packed codes and scales.  A workgroup takes 64 columns x 128 k, a wave 16 of the columns, a lane one block of 32 k:
// its 16 bytes of codes are that lane's MFMA operand, so that a wave writes 1 KiB in one piece, and no lane needs another's
// maximum.  The four waves' scale bytes meet in LDS and go out as 256 bytes.  DT -1: the codes exist, W holds them row by row.
template <int DT>
__global__ __launch_bounds__(256) void mx_pack_kernel(const uint8_t* W, const uint8_t* S, int N, int K, long long ldw, long long lds,
                                                      long long expert_stride, int cols, uint8_t* blob, long long blob_stride,
                                                      MxLayout L) {
    constexpr int ES = DT == W4A8_F32 ? 4 : 2;
    __shared__ uint8_t bytes[256];
    const int lane = int(threadIdx.x) & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const long long item = (long long)blockIdx.x / L.K1;
    const int step = int((long long)blockIdx.x - item * L.K1);
    const long long e = item / cols;
    const int cb = int(item - e * cols), n = cb * 64 + wave * 16 + (lane & 15), k = step * MX_STEP + (lane >> 4) * 32;
    uint8_t* out = blob + size_t(e) * size_t(blob_stride);
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    uint32_t byte = 0;
    if (n < N && k < K) {
        if constexpr (DT < 0) {
            q = *reinterpret_cast<const uint4*>(W + size_t(n) * size_t(ldw) + size_t(k) / 2);
            byte = S[size_t(n) * size_t(lds) + size_t(k) / 32];
        } else {
            const uint8_t* row = W + (size_t(e) * size_t(expert_stride) + size_t(n) * size_t(ldw)) * ES;
            float v[4][8];
            uint32_t amax = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mx_load8<DT>(row + size_t(min(k + 8 * i, K)) * ES, K - k - 8 * i, v[i]);
                amax = max(amax, mx_amax8(v[i]));
            }
            byte = mx_scale_byte<W4A8_MX_FP4>(amax);
            q = make_uint4(mx_encode8<W4A8_MX_FP4>(v[0], byte).x, mx_encode8<W4A8_MX_FP4>(v[1], byte).x,
                           mx_encode8<W4A8_MX_FP4>(v[2], byte).x, mx_encode8<W4A8_MX_FP4>(v[3], byte).x);
        }
    }
    if (cb * 64 + wave * 16 < N)                                // whole 16-column tiles that the blob has
        *reinterpret_cast<uint4*>(out + (size_t(cb * 4 + wave) * size_t(L.K1) + size_t(step)) * 1024 + lane * 16) = q;
    bytes[lane * 4 + wave] = uint8_t(byte);
    __syncthreads();
    if (wave == 0)
        *reinterpret_cast<uint32_t*>(out + L.scales_off + (size_t(cb) * size_t(L.K1) + size_t(step)) * 256 + lane * 4) =
            *reinterpret_cast<const uint32_t*>(bytes + lane * 4);
}

// Packed weights -> codes and scales row by row.
__global__ __launch_bounds__(256) void mx_unpack_kernel(const uint8_t* blob, MxLayout L, int N, int K, uint8_t* W, uint8_t* S) {
    const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
    const int cb = int(blockIdx.x / unsigned(L.K1)), step = int(blockIdx.x % unsigned(L.K1));
    const int n = cb * 64 + wave * 16 + (lane & 15), k = step * MX_STEP + (lane >> 4) * 32;
    if (n >= N) return;
    const int Kp = L.K1 * MX_STEP;
    *reinterpret_cast<uint4*>(W + size_t(n) * size_t(Kp / 2) + size_t(k) / 2) =
        *reinterpret_cast<const uint4*>(blob + (size_t(cb * 4 + wave) * size_t(L.K1) + size_t(step)) * 1024 + lane * 16);
    S[size_t(n) * size_t(Kp / 32) + size_t(k) / 32] =
        blob[L.scales_off + (size_t(cb) * size_t(L.K1) + size_t(step)) * 256 + lane * 4 + wave];
}

// Limits of the calls: rows and columns below 2^24, K below 2^20 (32-bit offsets within a row's chunks and a tile's steps).
static bool mx_fmt(int fmt) { return fmt == W4A8_MX_FP4 || fmt == W4A8_MX_FP8; }
static bool mx_type(int dt) { return dt == W4A8_BF16 || dt == W4A8_F16 || dt == W4A8_F32; }
static bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
static int launched() { return hipGetLastError() == hipSuccess ? W4A8_OK : W4A8_EHIP; }

template <int DT>
static void launch_quant(const void* X, int M, int K, int ldx, int fmt, void* Xq, uint8_t* sx, hipStream_t s) {
    const int chunks = (mx_kp(K) + 511) / 512;
    const dim3 grid(unsigned(((long long)M * chunks + 3) / 4));
    const uint8_t* x = static_cast<const uint8_t*>(X);
    uint8_t* q = static_cast<uint8_t*>(Xq);
    if (fmt == W4A8_MX_FP4) mx_quant_kernel<DT, W4A8_MX_FP4><<<grid, dim3(256), 0, s>>>(x, M, K, ldx, chunks, q, sx);
    else mx_quant_kernel<DT, W4A8_MX_FP8><<<grid, dim3(256), 0, s>>>(x, M, K, ldx, chunks, q, sx);
}

void launch_route_quant(const int32_t* ids, int R, int E, int32_t* rows, int32_t* offs, int32_t* inv, const void* X, int M, int K,
                        int fmt, uint8_t* Xq, uint8_t* sx, hipStream_t s) {
    const int chunks = (mx_kp(K) + 511) / 512;
    const dim3 grid(unsigned((E + 3) / 4 + ((long long)M * chunks + 3) / 4));
    const uint8_t* x = static_cast<const uint8_t*>(X);
    if (fmt == W4A8_MX_FP4) mx_route_quant_kernel<W4A8_MX_FP4><<<grid, dim3(256), 0, s>>>(ids, R, E, rows, offs, inv, x, M, K, chunks, Xq, sx);
    else mx_route_quant_kernel<W4A8_MX_FP8><<<grid, dim3(256), 0, s>>>(ids, R, E, rows, offs, inv, x, M, K, chunks, Xq, sx);
}

template <int FMT>
static void launch_dequant(const void* Xq, const uint8_t* sx, int M, int K, void* Y, int dtype, int ldy, hipStream_t s) {
    const int chunks = (K + 511) / 512;
    const dim3 grid(unsigned(((long long)M * chunks + 3) / 4));
    const uint8_t* q = static_cast<const uint8_t*>(Xq);
    uint8_t* y = static_cast<uint8_t*>(Y);
    if (dtype == W4A8_BF16) mx_dequant_kernel<FMT, W4A8_BF16><<<grid, dim3(256), 0, s>>>(q, sx, M, K, chunks, y, ldy);
    else if (dtype == W4A8_F16) mx_dequant_kernel<FMT, W4A8_F16><<<grid, dim3(256), 0, s>>>(q, sx, M, K, chunks, y, ldy);
    else mx_dequant_kernel<FMT, W4A8_F32><<<grid, dim3(256), 0, s>>>(q, sx, M, K, chunks, y, ldy);
}

// A launch has less than 2^32 work-items: fewer than 2^24 workgroups of 256.
constexpr long long MX_MAX_BLOCKS = (1ll << 24) - 1;

static int check_rows(const void* a, const void* b, const void* c, int fmt, int dtype, int M, int K, int ld) {
    if (!mx_fmt(fmt) || !mx_type(dtype) || M < 0 || K <= 0 || ld < K) return W4A8_EINVAL;
    if (K > MX_MAX_K || ((long long)M * ((mx_kp(K) + 511) / 512) + 3) / 4 > MX_MAX_BLOCKS) return W4A8_EUNSUPPORTED;
    if (M == 0) return W4A8_OK;
    return a && b && c ? W4A8_OK : W4A8_EINVAL;
}

static int check_weights(int N, int K) {
    if (N <= 0 || K <= 0) return W4A8_EINVAL;
    if (K > MX_MAX_K || N > MX_MAX_N || mx_layout(N, K).codes_bytes >= (size_t(1) << 31)) return W4A8_EUNSUPPORTED;
    return W4A8_OK;
}

int mx_check_weights(int N, int K) { return check_weights(N, K); }

}  // namespace w4a8

using namespace w4a8;

extern "C" {

int w4a8_mx_quant(const void* X, int dtype, int M, int K, int ldx, int fmt, void* Xq, uint8_t* sx, void* stream) {
    const int st = check_rows(X, Xq, sx, fmt, dtype, M, K, ldx);
    if (st || M == 0) return st;
    if (!aligned_to(X, dtype == W4A8_F32 ? 4 : 2) || !aligned_to(Xq, 16) || !aligned_to(sx, 4)) return W4A8_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == W4A8_BF16) launch_quant<W4A8_BF16>(X, M, K, ldx, fmt, Xq, sx, s);
    else if (dtype == W4A8_F16) launch_quant<W4A8_F16>(X, M, K, ldx, fmt, Xq, sx, s);
    else launch_quant<W4A8_F32>(X, M, K, ldx, fmt, Xq, sx, s);
    return launched();
}

int w4a8_mx_dequant(const void* Xq, const uint8_t* sx, int fmt, int M, int K, void* Y, int dtype, int ldy, void* stream) {
    const int st = check_rows(Y, Xq, sx, fmt, dtype, M, K, ldy);
    if (st || M == 0) return st;
    if (!aligned_to(Y, dtype == W4A8_F32 ? 4 : 2) || !aligned_to(Xq, 16) || !aligned_to(sx, 4)) return W4A8_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (fmt == W4A8_MX_FP4) launch_dequant<W4A8_MX_FP4>(Xq, sx, M, K, Y, dtype, ldy, s);
    else launch_dequant<W4A8_MX_FP8>(Xq, sx, M, K, Y, dtype, ldy, s);
    return launched();
}

size_t w4a8_mx_packed_size(int K, int N) { return check_weights(N, K) ? 0 : mx_layout(N, K).total; }

int w4a8_mx_pack(const void* W, int dtype, int E, int N, int K, int ldw, size_t expert_stride, void* blobs, size_t blob_stride,
                 void* stream) {
    int st = check_weights(N, K);
    if (st) return st;
    if (!mx_type(dtype) || E < 0 || E > 1024 || ldw < K) return W4A8_EINVAL;
    if (E == 0) return W4A8_OK;
    const MxLayout L = mx_layout(N, K);
    if (!W || !blobs || !aligned_to(W, dtype == W4A8_F32 ? 4 : 2) || !aligned_to(blobs, 16) || (blob_stride & 15)) return W4A8_EINVAL;
    if (E > 1 && (blob_stride < L.total || expert_stride < size_t(N - 1) * size_t(ldw) + size_t(K))) return W4A8_EINVAL;
    if (expert_stride > (size_t(1) << 60) || blob_stride > (size_t(1) << 60)) return W4A8_EINVAL;
    const int cols = (N + 63) / 64;
    const long long blocks = (long long)E * cols * L.K1;
    if (blocks > MX_MAX_BLOCKS) return W4A8_EUNSUPPORTED;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const uint8_t* w = static_cast<const uint8_t*>(W);
    uint8_t* b = static_cast<uint8_t*>(blobs);
    const dim3 grid(static_cast<unsigned>(blocks));
    const long long es = (long long)expert_stride, bs = (long long)blob_stride;
    if (dtype == W4A8_BF16) mx_pack_kernel<W4A8_BF16><<<grid, dim3(256), 0, s>>>(w, nullptr, N, K, ldw, 0, es, cols, b, bs, L);
    else if (dtype == W4A8_F16) mx_pack_kernel<W4A8_F16><<<grid, dim3(256), 0, s>>>(w, nullptr, N, K, ldw, 0, es, cols, b, bs, L);
    else mx_pack_kernel<W4A8_F32><<<grid, dim3(256), 0, s>>>(w, nullptr, N, K, ldw, 0, es, cols, b, bs, L);
    return launched();
}

int w4a8_mx_pack_codes(const uint8_t* codes, const uint8_t* scales, int N, int K, int ldc, int lds, void* blob, void* stream) {
    const int st = check_weights(N, K);
    if (st) return st;
    if (K % 32 || ldc < K / 2 || ldc % 16 || lds < K / 32) return W4A8_EINVAL;
    if (!codes || !scales || !blob || !aligned_to(codes, 16) || !aligned_to(blob, 16)) return W4A8_EINVAL;
    const MxLayout L = mx_layout(N, K);
    const int cols = (N + 63) / 64;
    if ((long long)cols * L.K1 > MX_MAX_BLOCKS) return W4A8_EUNSUPPORTED;
    mx_pack_kernel<-1><<<dim3(unsigned(cols * L.K1)), dim3(256), 0, static_cast<hipStream_t>(stream)>>>(
        codes, scales, N, K, ldc, lds, 0, cols, static_cast<uint8_t*>(blob), 0, L);
    return launched();
}

int w4a8_mx_unpack_codes(const void* blob, int N, int K, uint8_t* codes, uint8_t* scales, void* stream) {
    const int st = check_weights(N, K);
    if (st) return st;
    if (!blob || !codes || !scales || !aligned_to(blob, 16) || !aligned_to(codes, 16)) return W4A8_EINVAL;
    const MxLayout L = mx_layout(N, K);
    const int cols = (N + 63) / 64;
    if ((long long)cols * L.K1 > MX_MAX_BLOCKS) return W4A8_EUNSUPPORTED;
    mx_unpack_kernel<<<dim3(unsigned(cols * L.K1)), dim3(256), 0, static_cast<hipStream_t>(stream)>>>(
        static_cast<const uint8_t*>(blob), L, N, K, codes, scales);
    return launched();
}

}  // extern "C"
