// Tokens sorted by expert and back, with the routes' weights, and the
// gradients: a user's own experts (or their backward pass) on moe_route's maps,
// beside the expert step, which gathers its rows by itself, and moe_finalize,
// which norms each row on the way back.
//
//   moe_dispatch      rows[p(t,k)] = x[t]                     p = exp2perm, absent routes skipped
//   moe_dispatch_bwd  d_x[t] = sum_k d_rows[p(t,k)]
//   moe_combine       out[t] = sum_k w[t,k] rows[p(t,k)]
//   moe_combine_bwd   d_rows[p(t,k)] = w[t,k] d_out[t];  d_w[t,k] = <rows[p(t,k)], d_out[t]>
//
// All four are HBM-bound: each routed row moves once, each token row once. The
// token-to-rows calls walk the tokens, not the rows: a token's row is read into
// registers and written K times (walking the rows would read it K times). The
// rows-to-token calls issue the loads of 8 routes together and add them in
// route order in fp32, so the results are deterministic. No atomics.
#include "common.hpp"

namespace moe {

constexpr int kPadRows = 16;        // permuted rows a padding workgroup looks at (tiles are multiples of 16)
constexpr int kSortBatch = 8;       // routes whose loads issue together
// moe_combine_bwd: below so many 16-byte units of token rows (1 MiB) a workgroup
// takes one route instead of one token, for more rows in flight. Top-8, split
// and not: rows of 8 KiB, 8 tokens 4.5 and 6.6 us, 64 5.6 and 7.1, 128 7.8 and
// 7.8, 256 12.0 and 10.5; of 2 KiB, 256 tokens 5.2 and 6.1, 512 7.7 and 7.7;
// of 16 KiB, 64 tokens 10.3 and 10.8, 128 12.8 and 11.9. moe_dispatch gains
// nothing by it (8 tokens 4.8 and 4.7 us).
constexpr int64_t kRouteSplitUnits = 65536;

struct SortArgs {
    const uint8_t* tok;             // token rows: x, or d_out
    int64_t tok_stride;             // bytes
    const uint8_t* rows_in;         // moe_combine_bwd: the experts' rows
    int64_t rows_in_stride;
    const int32_t* exp2perm;
    const int32_t* perm2tok;
    const int32_t* total_rows;
    const float* weights;
    int T, K;
    int64_t R;                      // rows_max
    int units;                      // 16-byte units per row
    uint8_t* rows;
    int64_t rows_stride;
    float* d_weights;
    int work_groups;                // workgroups before the padding ones
    int col_groups;                 // workgroups a token or route is split into
};

__device__ __forceinline__ uint4 load16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
// Non-temporal: the rows written are far more than an L2 holds, and without it
// they displace the rows read (4096 tokens x 4096 bf16, top-8 of 128 experts:
// moe_dispatch 107.8 -> 65.4 us, moe_combine_bwd 176.1 -> 129.2, moe_combine
// 64.1 -> 57.3; from 1 to 512 tokens the same or up to 30% less).
__device__ __forceinline__ void store16(uint8_t* p, uint4 v) { store_stream16(p, v); }

// A route's permuted row, or -1 (absent, or outside the rows).
__device__ __forceinline__ int64_t route_row(const int32_t* exp2perm, int64_t route, int64_t R) {
    const int32_t p = exp2perm[route];
    return p >= 0 && p < R ? (int64_t)p : -1;
}

// The rows of one group of kPadRows that hold no route though they lie below
// total_rows (the ends of the experts' tiles): zeros, so that products over
// whole tiles of the rows, the weights' gradients among them, are the routes'
// alone. Rows from total_rows on are left as they were.
__device__ __forceinline__ void zero_padding(const SortArgs& a, int64_t group) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int64_t total = *a.total_rows, p0 = group * kPadRows, p = p0 + lane;
    // one load looks at the group's rows, a wave then takes every waves-th
    bool empty = false;
    if (lane < kPadRows && p < a.R && p < total) empty = a.perm2tok[p] < 0;
    uint64_t rows = __ballot(empty);
    for (int n = 0; rows; ++n, rows &= rows - 1) {
        if (n % waves != wave) continue;
        uint8_t* row = a.rows + (p0 + __builtin_ctzll(rows)) * a.rows_stride;
        for (int u = lane; u < a.units; u += 64) store16(row + (int64_t)u * 16, make_uint4(0u, 0u, 0u, 0u));
    }
}

// moe_dispatch: a workgroup copies 256 units of one token's row to the rows of
// all its routes.
__global__ void __launch_bounds__(256) dispatch_kernel(SortArgs a) {
    if ((int)blockIdx.x >= a.work_groups) return zero_padding(a, (int)blockIdx.x - a.work_groups);
    const int t = blockIdx.x / a.col_groups, c = blockIdx.x - t * a.col_groups;
    const int u = c * (int)blockDim.x + threadIdx.x;
    if (u >= a.units) return;
    const uint4 v = load16(a.tok + t * a.tok_stride + (int64_t)u * 16);
    for (int k = 0; k < a.K; ++k) {
        const int64_t p = route_row(a.exp2perm, (int64_t)t * a.K + k, a.R);
        if (p >= 0) store16(a.rows + p * a.rows_stride + (int64_t)u * 16, v);
    }
}

// ------------------------------------------------------------------ 16-byte units as fp32
template <bool kF32>
struct Unit {
    static constexpr int kN = kF32 ? 4 : 8;
    __device__ static __forceinline__ void unpack(const uint4& p, float (&v)[kN]) {
        const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kF32) {
                v[i] = __uint_as_float(w[i]);
            } else {
                v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
    __device__ static __forceinline__ uint4 pack(const float (&v)[kN]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kF32) w[i] = __float_as_uint(v[i]);
            else w[i] = f32_to_bf16(v[2 * i]) | (f32_to_bf16(v[2 * i + 1]) << 16);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// moe_combine (weights) and moe_dispatch_bwd (weights NULL: ones): a thread
// owns one unit of one token's output.
template <bool kF32>
__global__ void __launch_bounds__(256) combine_kernel(SortArgs a) {
    constexpr int n = Unit<kF32>::kN;
    const int t = blockIdx.x / a.col_groups, c = blockIdx.x - t * a.col_groups;
    const int u = c * (int)blockDim.x + threadIdx.x;
    if (u >= a.units) return;
    float acc[n];
#pragma unroll
    for (int i = 0; i < n; ++i) acc[i] = 0.0f;
    for (int k0 = 0; k0 < a.K; k0 += kSortBatch) {
        uint4 raw[kSortBatch];
        int64_t p[kSortBatch];
#pragma unroll
        for (int kk = 0; kk < kSortBatch; ++kk)
            p[kk] = k0 + kk < a.K ? route_row(a.exp2perm, (int64_t)t * a.K + k0 + kk, a.R) : -1;
#pragma unroll
        for (int kk = 0; kk < kSortBatch; ++kk)
            if (p[kk] >= 0) raw[kk] = load16(a.rows_in + p[kk] * a.rows_in_stride + (int64_t)u * 16);
#pragma unroll
        for (int kk = 0; kk < kSortBatch; ++kk) {
            if (p[kk] < 0) continue;
            const float w = a.weights ? a.weights[(int64_t)t * a.K + k0 + kk] : 1.0f;
            float v[n];
            Unit<kF32>::unpack(raw[kk], v);
#pragma unroll
            for (int i = 0; i < n; ++i) acc[i] = __fmaf_rn(w, v[i], acc[i]);
        }
    }
    store16(a.rows + t * a.rows_stride + (int64_t)u * 16, Unit<kF32>::pack(acc));
}

// moe_combine_bwd: a workgroup holds one token's d_out row in registers (NU
// units a thread) for all its routes, or (kSplit) for one; batches of B routes
// whose row loads issue together (4096 tokens, top-8, rows of 8 KiB: NU = 1 and
// B = 8 121.4 us, 2 and 4 129.0, 2 and 8 122.6; 512 tokens 15.7, 16.0, 16.2). The weight's gradient is a sum over the row:
// per thread in fp32, then over the wave, then over the waves in order.
template <bool kF32, int NU, int B, bool kSplit>
__global__ void __launch_bounds__(1024) combine_bwd_kernel(SortArgs a) {
    constexpr int n = Unit<kF32>::kN;
    __shared__ float s_dot[B][16];
    if ((int)blockIdx.x >= a.work_groups) return zero_padding(a, (int)blockIdx.x - a.work_groups);
    const int t = kSplit ? blockIdx.x / a.K : blockIdx.x;
    const int first = kSplit ? (int)blockIdx.x - t * a.K : 0, last = kSplit ? first + 1 : a.K;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
    uint4 g[NU];
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        const int u = tid + j * (int)blockDim.x;
        g[j] = u < a.units ? load16(a.tok + t * a.tok_stride + (int64_t)u * 16) : make_uint4(0u, 0u, 0u, 0u);
    }
    for (int k0 = first; k0 < last; k0 += B) {
        uint4 raw[B][NU];
        int64_t p[B];
#pragma unroll
        for (int kk = 0; kk < B; ++kk)
            p[kk] = k0 + kk < last ? route_row(a.exp2perm, (int64_t)t * a.K + k0 + kk, a.R) : -1;
#pragma unroll
        for (int kk = 0; kk < B; ++kk)
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                const int u = tid + j * (int)blockDim.x;
                if (p[kk] >= 0 && u < a.units)
                    raw[kk][j] = load16(a.rows_in + p[kk] * a.rows_in_stride + (int64_t)u * 16);
            }
#pragma unroll
        for (int kk = 0; kk < B; ++kk) {
            float dot = 0.0f;
            if (p[kk] >= 0) {
                const float w = a.weights[(int64_t)t * a.K + k0 + kk];
#pragma unroll
                for (int j = 0; j < NU; ++j) {
                    const int u = tid + j * (int)blockDim.x;
                    if (u >= a.units) continue;
                    float d[n], v[n];
                    Unit<kF32>::unpack(g[j], d);
                    Unit<kF32>::unpack(raw[kk][j], v);
#pragma unroll
                    for (int i = 0; i < n; ++i) {
                        dot = __fmaf_rn(d[i], v[i], dot);
                        d[i] = __fmul_rn(w, d[i]);
                    }
                    store16(a.rows + p[kk] * a.rows_stride + (int64_t)u * 16, Unit<kF32>::pack(d));
                }
            }
            dot = wave_sum(dot);
            if (lane == 0) s_dot[kk][wave] = dot;
        }
        __syncthreads();
        if (tid < B && k0 + tid < last) {
            float sum = 0.0f;
            for (int w = 0; w < waves; ++w) sum = __fadd_rn(sum, s_dot[tid][w]);
            a.d_weights[(int64_t)t * a.K + k0 + tid] = sum;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ host side
static int sort_sizes(int T, int K, int64_t rows_max, const char* name) {
    if (T < 0 || K < 1 || K > MOE_MAX_TOPK || rows_max < 0 || rows_max > 0x7FFFFFFF)
        return fail(MOE_EINVAL, "%s: T=%d K=%d rows_max=%lld out of range", name, T, K, (long long)rows_max);
    if ((int64_t)T * K > 0x7FFFFFFF) return fail(MOE_EUNSUPPORTED, "%s: too many routes", name);
    return MOE_OK;
}

static int typed_row(int dtype, int H, const char* name) {
    if (dtype != MOE_BF16 && dtype != MOE_F32)
        return fail(MOE_EINVAL, "%s: dtype %d is neither MOE_BF16 nor MOE_F32", name, dtype);
    if (H < 0) return fail(MOE_EINVAL, "%s: negative size H=%d", name, H);
    if (H % 8 || H > MOE_MAX_HIDDEN)
        return fail(MOE_EUNSUPPORTED, "%s: H=%d must be a multiple of 8 up to %d", name, H, MOE_MAX_HIDDEN);
    return MOE_OK;
}

static bool bad_stride(int64_t stride, int H) { return stride < H || stride % 8; }

// rows -> tokens, shared by moe_combine and moe_dispatch_bwd
static int launch_combine(const void* rows, int64_t rows_stride, int dtype, const int32_t* exp2perm,
                          const float* weights, int T, int K, int64_t rows_max, int H, void* out,
                          int64_t out_row_stride, void* stream, const char* name) {
    const int es = dtype == MOE_F32 ? 4 : 2;
    if (!rows || !exp2perm || !out) return fail(MOE_EINVAL, "%s: NULL pointer", name);
    if (!aligned16(rows) || !aligned16(exp2perm) || !aligned16(out) || !aligned16(weights))
        return fail(MOE_EINVAL, "%s: pointers must be 16-byte aligned", name);
    if (bad_stride(rows_stride, H) || bad_stride(out_row_stride, H))
        return fail(MOE_EINVAL, "%s: row strides must be >= H and multiples of 8", name);
    SortArgs a{};
    a.rows_in = (const uint8_t*)rows; a.rows_in_stride = rows_stride * es;
    a.exp2perm = exp2perm; a.weights = weights; a.T = T; a.K = K; a.R = rows_max;
    a.units = H * es / 16; a.rows = (uint8_t*)out; a.rows_stride = out_row_stride * es;
    // 64-thread workgroups while there is less than one of 256 threads a CU (8192
    // bytes a token: 64 tokens 4.2 us against 4.4, 128 tokens 5.4 against 4.9)
    const int threads = (int64_t)T * ((a.units + 255) / 256) >= 256 ? 256 : 64;
    a.col_groups = (a.units + threads - 1) / threads;
    const int64_t grid = (int64_t)T * a.col_groups;
    if (!launch_fits(grid, threads)) return fail(MOE_EUNSUPPORTED, "%s: too large", name);
    const dim3 g((unsigned)grid), b((unsigned)threads);
    if (dtype == MOE_F32) hipLaunchKernelGGL(combine_kernel<true>, g, b, 0, (hipStream_t)stream, a);
    else hipLaunchKernelGGL(combine_kernel<false>, g, b, 0, (hipStream_t)stream, a);
    return check_launch(name);
}

// A thread a unit up to 1024 threads, then 2 or 4 units a thread.
static int bwd_threads(int units) { return units < 1024 ? (units + 63) / 64 * 64 : 1024; }

template <bool kF32>
void launch_combine_bwd(const SortArgs& a, unsigned grid, bool split, hipStream_t s) {
    const dim3 g(grid), b((unsigned)bwd_threads(a.units));
    if (a.units <= 1024) {
        if (split) hipLaunchKernelGGL((combine_bwd_kernel<kF32, 1, 1, true>), g, b, 0, s, a);
        else hipLaunchKernelGGL((combine_bwd_kernel<kF32, 1, 8, false>), g, b, 0, s, a);
    } else if (a.units <= 2048) {
        if (split) hipLaunchKernelGGL((combine_bwd_kernel<kF32, 2, 1, true>), g, b, 0, s, a);
        else hipLaunchKernelGGL((combine_bwd_kernel<kF32, 2, 4, false>), g, b, 0, s, a);
    } else {
        if (split) hipLaunchKernelGGL((combine_bwd_kernel<kF32, 4, 1, true>), g, b, 0, s, a);
        else hipLaunchKernelGGL((combine_bwd_kernel<kF32, 4, 2, false>), g, b, 0, s, a);
    }
}

}  // namespace moe

extern "C" int moe_dispatch(const void* x, int64_t x_row_stride_bytes, int64_t row_bytes, const int32_t* exp2perm,
                            const int32_t* perm2tok, const int32_t* total_rows, int T, int K, int64_t rows_max,
                            void* rows, int64_t rows_stride_bytes, void* stream) {
    using namespace moe;
    const char* name = "moe_dispatch";
    const int rc = sort_sizes(T, K, rows_max, name);
    if (rc != MOE_OK) return rc;
    if (row_bytes < 0 || row_bytes % 16 || row_bytes > 4LL * MOE_MAX_HIDDEN)
        return fail(MOE_EUNSUPPORTED, "%s: row_bytes=%lld must be a multiple of 16 up to %d", name,
                    (long long)row_bytes, 4 * MOE_MAX_HIDDEN);
    if (T == 0 || row_bytes == 0) return MOE_OK;
    if (!x || !exp2perm || !perm2tok || !total_rows || !rows) return fail(MOE_EINVAL, "%s: NULL pointer", name);
    if (!aligned16(x) || !aligned16(exp2perm) || !aligned16(perm2tok) || !aligned16(rows) ||
        (reinterpret_cast<uintptr_t>(total_rows) & 3u))
        return fail(MOE_EINVAL, "%s: pointers must be 16-byte aligned (total_rows: 4)", name);
    if (x_row_stride_bytes < row_bytes || x_row_stride_bytes % 16 || rows_stride_bytes < row_bytes ||
        rows_stride_bytes % 16)
        return fail(MOE_EINVAL, "%s: row strides must be >= row_bytes and multiples of 16", name);
    SortArgs a{};
    a.tok = (const uint8_t*)x; a.tok_stride = x_row_stride_bytes; a.exp2perm = exp2perm; a.perm2tok = perm2tok;
    a.total_rows = total_rows; a.T = T; a.K = K; a.R = rows_max; a.units = (int)(row_bytes / 16);
    a.rows = (uint8_t*)rows; a.rows_stride = rows_stride_bytes;
    a.col_groups = (a.units + 255) / 256;
    const int64_t work = (int64_t)T * a.col_groups, pad = (rows_max + kPadRows - 1) / kPadRows;
    if (!launch_fits(work + pad, 256)) return fail(MOE_EUNSUPPORTED, "%s: too large", name);
    a.work_groups = (int)work;
    const dim3 g((unsigned)(work + pad)), b(256);
    hipLaunchKernelGGL(dispatch_kernel, g, b, 0, (hipStream_t)stream, a);
    return check_launch(name);
}

extern "C" int moe_dispatch_bwd(const void* d_rows, int64_t rows_stride, int dtype, const int32_t* exp2perm, int T,
                                int K, int64_t rows_max, int H, void* d_x, int64_t d_x_row_stride, void* stream) {
    using namespace moe;
    const char* name = "moe_dispatch_bwd";
    int rc = sort_sizes(T, K, rows_max, name);
    if (rc == MOE_OK) rc = typed_row(dtype, H, name);
    if (rc != MOE_OK || T == 0 || H == 0) return rc;
    return launch_combine(d_rows, rows_stride, dtype, exp2perm, nullptr, T, K, rows_max, H, d_x, d_x_row_stride, stream,
                          name);
}

extern "C" int moe_combine(const void* rows, int64_t rows_stride, int dtype, const int32_t* exp2perm,
                           const float* topk_weights, int T, int K, int64_t rows_max, int H, void* out,
                           int64_t out_row_stride, void* stream) {
    using namespace moe;
    const char* name = "moe_combine";
    int rc = sort_sizes(T, K, rows_max, name);
    if (rc == MOE_OK) rc = typed_row(dtype, H, name);
    if (rc != MOE_OK || T == 0 || H == 0) return rc;
    if (!topk_weights) return fail(MOE_EINVAL, "%s: NULL pointer", name);
    return launch_combine(rows, rows_stride, dtype, exp2perm, topk_weights, T, K, rows_max, H, out, out_row_stride,
                          stream, name);
}

extern "C" int moe_combine_bwd(const void* d_out, int64_t d_out_row_stride, const void* rows, int64_t rows_stride,
                               int dtype, const int32_t* exp2perm, const int32_t* perm2tok, const int32_t* total_rows,
                               const float* topk_weights, int T, int K, int64_t rows_max, int H, void* d_rows,
                               int64_t d_rows_stride, float* d_weights, void* stream) {
    using namespace moe;
    const char* name = "moe_combine_bwd";
    int rc = sort_sizes(T, K, rows_max, name);
    if (rc == MOE_OK) rc = typed_row(dtype, H, name);
    if (rc != MOE_OK || T == 0 || H == 0) return rc;
    if (!d_out || !rows || !exp2perm || !perm2tok || !total_rows || !topk_weights || !d_rows || !d_weights)
        return fail(MOE_EINVAL, "%s: NULL pointer", name);
    if (!aligned16(d_out) || !aligned16(rows) || !aligned16(exp2perm) || !aligned16(perm2tok) ||
        !aligned16(topk_weights) || !aligned16(d_rows) || !aligned16(d_weights) ||
        (reinterpret_cast<uintptr_t>(total_rows) & 3u))
        return fail(MOE_EINVAL, "%s: pointers must be 16-byte aligned (total_rows: 4)", name);
    if (bad_stride(d_out_row_stride, H) || bad_stride(rows_stride, H) || bad_stride(d_rows_stride, H))
        return fail(MOE_EINVAL, "%s: row strides must be >= H and multiples of 8", name);
    if (d_rows == rows && d_rows_stride != rows_stride)
        return fail(MOE_EINVAL, "%s: d_rows in place of rows needs its row stride", name);
    const int es = dtype == MOE_F32 ? 4 : 2;
    SortArgs a{};
    a.tok = (const uint8_t*)d_out; a.tok_stride = d_out_row_stride * es;
    a.rows_in = (const uint8_t*)rows; a.rows_in_stride = rows_stride * es;
    a.exp2perm = exp2perm; a.perm2tok = perm2tok; a.total_rows = total_rows; a.weights = topk_weights;
    a.T = T; a.K = K; a.R = rows_max; a.units = H * es / 16;
    a.rows = (uint8_t*)d_rows; a.rows_stride = d_rows_stride * es; a.d_weights = d_weights;
    const bool split = (int64_t)T * a.units < kRouteSplitUnits;
    const int64_t work = (int64_t)T * (split ? K : 1), pad = (rows_max + kPadRows - 1) / kPadRows;
    if (!launch_fits(work + pad, bwd_threads(a.units))) return fail(MOE_EUNSUPPORTED, "%s: too large", name);
    a.work_groups = (int)work;
    if (dtype == MOE_F32) launch_combine_bwd<true>(a, (unsigned)(work + pad), split, (hipStream_t)stream);
    else launch_combine_bwd<false>(a, (unsigned)(work + pad), split, (hipStream_t)stream);
    return check_launch(name);
}
