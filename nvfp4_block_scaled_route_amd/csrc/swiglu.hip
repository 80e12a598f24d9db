// The gated activation between the two products grouped by expert, and its
// gradient, on rows sorted by moe_dispatch:
//   moe_swiglu      y = silu(g) u                       silu(g) = g s, s = 1 / (1 + exp(-g))
//   moe_swiglu_bwd  d_g = d_y u s (1 + g (1 - s));  d_u = d_y silu(g)
// g and u are the first and second half of a row of gate_up.
//
// Both are HBM-bound and move each byte once: a thread owns 16 bytes of g, u
// and y. 40704 rows of 1536 (32768 of them tokens'), bf16: the gradient 96 to 109 us,
// 4.6 to 5.2 TB/s of the 503 MB of the tokens' rows (a large copy 4.8); 64 tokens'
// rows forward 4.0 to 4.4 us, a launch. Padding rows below total_rows are written as zeros without being read,
// rows behind are left.
#include "common.hpp"

namespace moe {

struct SgArgs {
    const uint8_t* gate_up;
    const uint8_t* d_inter;     // the gradient alone
    const int32_t* perm2tok;
    const int32_t* total_rows;
    int64_t R;
    int64_t gate_up_stride, d_inter_stride, out_stride;     // bytes
    int units;                  // 16-byte units of I values
    uint8_t* out;
};

constexpr int kSgThreads = 256;

template <bool kF32>
struct SgUnit {
    static constexpr int kN = kF32 ? 4 : 8;
    __device__ static __forceinline__ void load(const uint8_t* p, float (&v)[kN]) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
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
    __device__ static __forceinline__ void store(uint8_t* p, const float (&v)[kN]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kF32) w[i] = __float_as_uint(v[i]);
            else w[i] = f32_to_bf16(v[2 * i]) | (f32_to_bf16(v[2 * i + 1]) << 16);
        }
        store_stream16(p, make_uint4(w[0], w[1], w[2], w[3]));
    }
};

// s = 1 / (1 + exp(-g)) and 1 - s, either without overflow or cancellation: with
// t = exp(-|g|) the larger is 1 / (1 + t) and the smaller t / (1 + t).
struct Sigmoid {
    float s, rest;
    __device__ __forceinline__ explicit Sigmoid(float g) {
        const float t = expf(-__builtin_fabsf(g)), large = __fdiv_rn(1.0f, __fadd_rn(1.0f, t)), small = __fmul_rn(t, large);
        s = g < 0.0f ? small : large;
        rest = g < 0.0f ? large : small;
    }
};

template <bool kF32, bool kBwd>
__global__ void __launch_bounds__(kSgThreads) swiglu_kernel(SgArgs a) {
    constexpr int n = SgUnit<kF32>::kN;
    const int64_t total = *a.total_rows < a.R ? *a.total_rows : a.R;
    // a workgroup's first unit by a uniform 64-bit division, a thread's by a 32-bit one
    const int64_t first = (int64_t)blockIdx.x * kSgThreads, row0 = first / a.units;
    const uint32_t o = (uint32_t)(first - row0 * a.units) + threadIdx.x, dr = o / (uint32_t)a.units;
    const int64_t row = row0 + dr, at = (int64_t)(o - dr * (uint32_t)a.units) * 16, half = (int64_t)a.units * 16;
    if (row >= total) return;
    uint8_t* out = a.out + row * a.out_stride + at;
    float g[n], u[n], y[n];
    if (a.perm2tok[row] < 0) {
#pragma unroll
        for (int i = 0; i < n; ++i) y[i] = 0.0f;
        SgUnit<kF32>::store(out, y);
        if constexpr (kBwd) SgUnit<kF32>::store(out + half, y);
        return;
    }
    const uint8_t* in = a.gate_up + row * a.gate_up_stride + at;
    SgUnit<kF32>::load(in, g);
    SgUnit<kF32>::load(in + half, u);
    if constexpr (!kBwd) {
#pragma unroll
        for (int i = 0; i < n; ++i) y[i] = __fmul_rn(__fmul_rn(g[i], Sigmoid(g[i]).s), u[i]);
        SgUnit<kF32>::store(out, y);
    } else {
        SgUnit<kF32>::load(a.d_inter + row * a.d_inter_stride + at, y);
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const Sigmoid z(g[i]);
            const float silu = __fmul_rn(g[i], z.s);
            // s (1 + g (1 - s)) = s + silu (1 - s)
            const float d_g = __fmul_rn(__fmul_rn(y[i], u[i]), __fmaf_rn(silu, z.rest, z.s));
            u[i] = __fmul_rn(y[i], silu);
            g[i] = d_g;
        }
        SgUnit<kF32>::store(out, g);
        SgUnit<kF32>::store(out + half, u);
    }
}

static int swiglu_call(const void* d_inter, int64_t d_inter_row_stride, const void* gate_up, int64_t gate_up_row_stride, int dtype,
                       const int32_t* perm2tok, const int32_t* total_rows, int64_t rows_max, int I, void* out,
                       int64_t out_row_stride, bool bwd, void* stream, const char* name) {
    if (rows_max < 0 || rows_max > 0x7FFFFFFF || I < 0)
        return fail(MOE_EINVAL, "%s: rows_max=%lld I=%d out of range", name, (long long)rows_max, I);
    if (dtype != MOE_BF16 && dtype != MOE_F32)
        return fail(MOE_EINVAL, "%s: dtype %d is neither MOE_BF16 nor MOE_F32", name, dtype);
    if (I % 8 || I > MOE_MAX_HIDDEN)
        return fail(MOE_EUNSUPPORTED, "%s: I=%d must be a multiple of 8 up to %d", name, I, MOE_MAX_HIDDEN);
    if (rows_max == 0 || I == 0) return MOE_OK;
    if (!gate_up || !out || !perm2tok || !total_rows || (bwd && !d_inter)) return fail(MOE_EINVAL, "%s: NULL pointer", name);
    if (!aligned16(gate_up) || !aligned16(out) || !aligned16(perm2tok) || !aligned16(d_inter) ||
        (reinterpret_cast<uintptr_t>(total_rows) & 3u))
        return fail(MOE_EINVAL, "%s: pointers must be 16-byte aligned (total_rows: 4)", name);
    const int64_t out_cols = bwd ? 2 * (int64_t)I : I;
    if (gate_up_row_stride < 2 * (int64_t)I || gate_up_row_stride % 8 || out_row_stride < out_cols || out_row_stride % 8 ||
        (bwd && (d_inter_row_stride < I || d_inter_row_stride % 8)))
        return fail(MOE_EINVAL, "%s: row strides must be >= the rows and multiples of 8", name);
    if (bwd && out == gate_up && out_row_stride != gate_up_row_stride)
        return fail(MOE_EINVAL, "%s: d_gate_up in place of gate_up needs its row stride", name);
    const int es = dtype == MOE_F32 ? 4 : 2;
    SgArgs a{(const uint8_t*)gate_up, (const uint8_t*)d_inter, perm2tok, total_rows, rows_max, gate_up_row_stride * es,
             d_inter_row_stride * es, out_row_stride * es, I * es / 16, (uint8_t*)out};
    const int64_t grid = (rows_max * a.units + kSgThreads - 1) / kSgThreads;
    if (!launch_fits(grid, kSgThreads)) return fail(MOE_EUNSUPPORTED, "%s: too large", name);
    const dim3 g((unsigned)grid), b(kSgThreads);
    hipStream_t s = (hipStream_t)stream;
    if (dtype == MOE_F32 && bwd) hipLaunchKernelGGL((swiglu_kernel<true, true>), g, b, 0, s, a);
    else if (dtype == MOE_F32) hipLaunchKernelGGL((swiglu_kernel<true, false>), g, b, 0, s, a);
    else if (bwd) hipLaunchKernelGGL((swiglu_kernel<false, true>), g, b, 0, s, a);
    else hipLaunchKernelGGL((swiglu_kernel<false, false>), g, b, 0, s, a);
    return check_launch(name);
}

}  // namespace moe

extern "C" int moe_swiglu(const void* gate_up, int64_t gate_up_row_stride, int dtype, const int32_t* perm2tok,
                          const int32_t* total_rows, int64_t rows_max, int I, void* inter, int64_t inter_row_stride, void* stream) {
    return moe::swiglu_call(nullptr, 0, gate_up, gate_up_row_stride, dtype, perm2tok, total_rows, rows_max, I, inter,
                            inter_row_stride, false, stream, "moe_swiglu");
}

extern "C" int moe_swiglu_bwd(const void* d_inter, int64_t d_inter_row_stride, const void* gate_up, int64_t gate_up_row_stride,
                              int dtype, const int32_t* perm2tok, const int32_t* total_rows, int64_t rows_max, int I,
                              void* d_gate_up, int64_t d_gate_up_row_stride, void* stream) {
    return moe::swiglu_call(d_inter, d_inter_row_stride, gate_up, gate_up_row_stride, dtype, perm2tok, total_rows, rows_max, I,
                            d_gate_up, d_gate_up_row_stride, true, stream, "moe_swiglu_bwd");
}
