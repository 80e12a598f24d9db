// The MX quantizer, its inverse, and the residual addition with RMSNorm whose
// output is MX: the activations of the dense products around the experts (the
// model page, "MuseSpark1xMoE": the pooler and unpooler projections; the
// residual boundary in front of them), in OCP microscaling formats.
//
//   mx_quant           x -> codes, e8m0 scales (per 32 values)
//   mx_dequant         codes, scales -> bf16 values
//   mx_add_norm_quant  h = bf16(x + residual); y = h / rms(h) * gain; MX(y)
//
// All three are HBM-bound and read and write each byte once. A lane owns 8
// values (one 16-byte bf16 load; 8 or 4 code bytes out), a quad one block: its
// amax is two DPP steps over the magnitudes' bits, no LDS.
#include "mx.hpp"

namespace moe {

constexpr int kMqThreads = 256;

struct MqArgs {
    const uint16_t* x;
    int64_t x_row_stride;
    int64_t octs;           // T * H / 8
    int row_octs;           // H / 8
    uint8_t* codes;
    uint8_t* sf;
};

// Octet i of the T x H values, row by row, in a matrix whose rows lie `stride`
// elements apart (ROWS: else rows follow one another and i is the place). A
// workgroup finds the row of its first octet once (a uniform 64-bit division),
// a lane its own by a 32-bit one. first is a multiple of 4 and H of 32, so quads
// hold whole blocks.
template <bool ROWS>
__device__ __forceinline__ int64_t octet_at(int64_t first, int off, int row_octs, int64_t stride) {
    if constexpr (!ROWS) return (first + off) * 8;
    const int64_t row0 = first / row_octs;
    const uint32_t o = (uint32_t)(first - row0 * row_octs) + (uint32_t)off, dr = o / (uint32_t)row_octs;
    return (row0 + dr) * stride + (int64_t)(o - dr * (uint32_t)row_octs) * 8;
}

// An octet a thread: 64 x 4096 2.7 us, 4096 x 4096 8.6 (e2m1) and 9.7 (e4m3), 16384 x 4096 30.7 and 36.6
// (5.5 TB/s); two a thread, or four, came to the same or 3% more at every size.
template <int FMT, bool ROWS>
__global__ void __launch_bounds__(kMqThreads) mx_quant_kernel(MqArgs a) {
    const int64_t first = (int64_t)blockIdx.x * kMqThreads, i = first + threadIdx.x;
    if (i >= a.octs) return;
    float v[8];
    unpack8(*reinterpret_cast<const uint4*>(a.x + octet_at<ROWS>(first, threadIdx.x, a.row_octs, a.x_row_stride)), v);
    mx_store8<FMT>(v, i, a.codes, a.sf);
}

struct MdArgs {
    const uint8_t* codes;
    const uint8_t* sf;
    int64_t octs;
    int row_octs;
    uint16_t* out;
    int64_t out_row_stride;
};

// code * 2^(byte - 127) in fp32 (exact; the factor of byte 0 is the subnormal
// 2^-127), rounded once to bf16; NaN under byte 255. An octet a thread; the
// output, the most of the bytes, is streamed: e2m1 4096 x 4096 10.5 -> 8.1 us,
// 16384 x 4096 48.9 -> 27.3 (6.2 TB/s), e4m3 46.4 -> 31.5 (6.4 TB/s).
template <int FMT, bool ROWS>
__global__ void __launch_bounds__(kMqThreads) mx_dequant_kernel(MdArgs a) {
    const int64_t first = (int64_t)blockIdx.x * kMqThreads, i = first + threadIdx.x;
    if (i >= a.octs) return;
    const uint32_t byte = a.sf[i >> 2];
    const float s = byte == 255u ? __uint_as_float(0x7FC00000u)
                                 : byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
    float v[8];
    if constexpr (FMT == MOE_MX_E2M1) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(a.codes + i * 4);
        // the hardware's conversion: e2m1 values are exact in f16
        const half2v h[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1),
                             __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3)};
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = (float)h[k / 2][k % 2];
    } else {
        // likewise, in fp32 at once; the NaN code becomes NaN
        const uint2 w = *reinterpret_cast<const uint2*>(a.codes + i * 8);
        const auto p0 = __builtin_amdgcn_cvt_pk_f32_fp8(w.x, false), p1 = __builtin_amdgcn_cvt_pk_f32_fp8(w.x, true),
                   p2 = __builtin_amdgcn_cvt_pk_f32_fp8(w.y, false), p3 = __builtin_amdgcn_cvt_pk_f32_fp8(w.y, true);
        v[0] = p0[0], v[1] = p0[1], v[2] = p1[0], v[3] = p1[1], v[4] = p2[0], v[5] = p2[1], v[6] = p3[0], v[7] = p3[1];
    }
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        o[k] = f32_to_bf16(__fmul_rn(v[2 * k], s)) | (f32_to_bf16(__fmul_rn(v[2 * k + 1], s)) << 16);
    store_stream16(a.out + octet_at<ROWS>(first, threadIdx.x, a.row_octs, a.out_row_stride), make_uint4(o[0], o[1], o[2], o[3]));
}

template <int FMT, bool ROWS>
void launch_quant(const MqArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((mx_quant_kernel<FMT, ROWS>), dim3((unsigned)((a.octs + kMqThreads - 1) / kMqThreads)),
                       dim3(kMqThreads), 0, s, a);
}

// ------------------------------------------------------------------ residual + norm + MX
struct AnArgs {
    const uint16_t* x;
    int64_t x_row_stride;
    const uint16_t* residual;       // or NULL
    int64_t residual_row_stride;
    const uint16_t* norm_weight;    // or NULL: ones
    float gain_center, eps;
    int T, H;
    uint16_t* sum;                  // or NULL (no residual)
    int64_t sum_row_stride;
    uint8_t* codes;
    uint8_t* sf;
};

__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
    return v;
}

// A workgroup of 64 to 1024 threads a row, NB octets a thread in registers from
// the load to the codes: one pass over memory, and a single token's row is in
// flight at once. The sum of squares is formed in fp64 (each square exact) and
// rounded once. (A wave a row without a barrier, for many rows, was slower:
// 4096 x 4096 30.5 us against 25.9 then, too little in flight at 8 octets a thread.)
template <int FMT, int NB>
__global__ void __launch_bounds__(1024) add_norm_kernel(AnArgs a) {
    __shared__ double s_part[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = blockIdx.x;
    const int first = threadIdx.x, step = blockDim.x;
    const int row_octs = a.H >> 3;
    uint4 h[NB], r[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int o = first + i * step;
        h[i] = r[i] = make_uint4(0u, 0u, 0u, 0u);
        if (o < row_octs) {
            h[i] = *reinterpret_cast<const uint4*>(a.x + t * a.x_row_stride + (int64_t)o * 8);
            if (a.residual)
                r[i] = *reinterpret_cast<const uint4*>(a.residual + t * a.residual_row_stride + (int64_t)o * 8);
        }
    }
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int o = first + i * step;
        if (o >= row_octs) continue;
        float v[8], w[8];
        unpack8(h[i], v);
        if (a.residual) {
            // the fp32 sum rounded to bf16, the residual stream's type: the norm
            // is of the values that the next layer will read
            unpack8(r[i], w);
            uint32_t b[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                b[k] = f32_to_bf16(__fadd_rn(v[k], w[k]));
                v[k] = bf16_to_f32(b[k]);
            }
            h[i] = make_uint4(b[0] | (b[1] << 16), b[2] | (b[3] << 16), b[4] | (b[5] << 16), b[6] | (b[7] << 16));
        }
        // streamed: the sum is read again a layer later (4096 x 4096 25.9 -> 21.4 us)
        if (a.sum) store_stream16(a.sum + t * a.sum_row_stride + (int64_t)o * 8, h[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = __fma_rn((double)v[k], (double)v[k], ss);
    }
    ss = wave_sum_d(ss);
    if (lane == 0) s_part[wave] = ss;
    __syncthreads();
    ss = 0.0;
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) ss += s_part[w];
    const double mean = __ddiv_rn(ss, (double)a.H);
    const float ms = __double2float_rn(mean);
    // sqrtf, not __fsqrt_rn: the latter is the bare v_sqrt_f32 here, which is off
    // by an ulp now and then
    const float rr = __fdiv_rn(1.0f, sqrtf(__fadd_rn(ms, a.eps)));
    const auto store = [&](auto norm) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int o = first + i * step;
            if (o >= row_octs) continue;
            float v[8], g[8];
            unpack8(h[i], v);
            if (a.norm_weight) unpack8(*reinterpret_cast<const uint4*>(a.norm_weight + (int64_t)o * 8), g);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = __fmul_rn(norm(v[k]), __fadd_rn(a.norm_weight ? g[k] : 1.0f, a.gain_center));
            mx_store8<FMT>(v, o, a.codes + t * mx_bytes(a.H, FMT), a.sf + t * (a.H >> 5));
        }
    };
    // A finite row may have a mean square past fp32's range (values above 1.8e19):
    // its reciprocal root is below fp32's normal numbers, so h * r is formed in
    // fp64 and rounded once. A branch of the wave: both ways for every element
    // cost 5% (4096 x 4096 21.0 -> 22.1 us). A row that holds an infinity is NaN
    // throughout, like one that holds a NaN: h / infinity would leave zeros, which
    // no later step tells from values.
    if (__builtin_amdgcn_readfirstlane(ms == INFINITY)) {
        const double rd = mean == (double)INFINITY ? (double)NAN : __ddiv_rn(1.0, sqrt(__dadd_rn(mean, (double)a.eps)));
        store([&](float x) { return __double2float_rn(__dmul_rn((double)x, rd)); });
    } else {
        store([&](float x) { return __fmul_rn(x, rr); });
    }
}

template <int FMT>
void launch_add_norm(const AnArgs& a, hipStream_t s) {
    const int octs = a.H >> 3;
    int threads = (octs + 63) / 64 * 64;
    if (threads > 1024) threads = 1024;
    const dim3 g((unsigned)a.T), b((unsigned)threads);
    if (octs <= 1024) hipLaunchKernelGGL((add_norm_kernel<FMT, 1>), g, b, 0, s, a);
    else hipLaunchKernelGGL((add_norm_kernel<FMT, 2>), g, b, 0, s, a);
}

// Sizes, format, alignment and strides of an MX conversion between [T, H] bf16
// rows and codes and scales.
static int mx_check(const void* x, int64_t x_row_stride, int T, int H, int fmt, const void* codes, const void* sf,
                    const char* name) {
    if (T < 0 || H < 0) return fail(MOE_EINVAL, "%s: negative size T=%d H=%d", name, T, H);
    if (!mx_fmt_ok(fmt)) return fail(MOE_EINVAL, "%s: format %d is neither MOE_MX_E2M1 nor MOE_MX_E4M3", name, fmt);
    if (H % kMxBlock) return fail(MOE_EUNSUPPORTED, "%s: H=%d is not a multiple of 32", name, H);
    if (T == 0 || H == 0) return MOE_OK;
    if (!x || !codes || !sf) return fail(MOE_EINVAL, "%s: NULL pointer", name);
    if (!aligned16(x) || !aligned16(codes) || !aligned16(sf))
        return fail(MOE_EINVAL, "%s: pointers must be 16-byte aligned", name);
    if (x_row_stride < H || x_row_stride % 8)
        return fail(MOE_EINVAL, "%s: row stride %lld must be >= H and a multiple of 8", name, (long long)x_row_stride);
    if (!launch_fits(((int64_t)T * (H / 8) + kMqThreads - 1) / kMqThreads, kMqThreads))
        return fail(MOE_EUNSUPPORTED, "%s: too large", name);
    return MOE_OK;
}

}  // namespace moe

extern "C" int mx_quant(const uint16_t* x, int64_t x_row_stride, int T, int H, int fmt, uint8_t* codes, uint8_t* sf,
                        void* stream) {
    using namespace moe;
    const int rc = mx_check(x, x_row_stride, T, H, fmt, codes, sf, "mx_quant");
    if (rc != MOE_OK || T == 0 || H == 0) return rc;
    MqArgs a{x, x_row_stride, (int64_t)T * (H / 8), H / 8, codes, sf};
    const bool rows = T > 1 && x_row_stride != H;
    if (fmt == MOE_MX_E2M1) rows ? launch_quant<MOE_MX_E2M1, true>(a, (hipStream_t)stream) : launch_quant<MOE_MX_E2M1, false>(a, (hipStream_t)stream);
    else rows ? launch_quant<MOE_MX_E4M3, true>(a, (hipStream_t)stream) : launch_quant<MOE_MX_E4M3, false>(a, (hipStream_t)stream);
    return check_launch("mx_quant");
}

extern "C" int mx_dequant(const uint8_t* codes, const uint8_t* sf, int T, int H, int fmt, uint16_t* out,
                          int64_t out_row_stride, void* stream) {
    using namespace moe;
    const int rc = mx_check(out, out_row_stride, T, H, fmt, codes, sf, "mx_dequant");
    if (rc != MOE_OK || T == 0 || H == 0) return rc;
    MdArgs a{codes, sf, (int64_t)T * (H / 8), H / 8, out, out_row_stride};
    const dim3 g((unsigned)((a.octs + kMqThreads - 1) / kMqThreads)), b(kMqThreads);
    hipStream_t st = (hipStream_t)stream;
    const bool rows = T > 1 && out_row_stride != H;
    if (fmt == MOE_MX_E2M1 && rows) hipLaunchKernelGGL((mx_dequant_kernel<MOE_MX_E2M1, true>), g, b, 0, st, a);
    else if (fmt == MOE_MX_E2M1) hipLaunchKernelGGL((mx_dequant_kernel<MOE_MX_E2M1, false>), g, b, 0, st, a);
    else if (rows) hipLaunchKernelGGL((mx_dequant_kernel<MOE_MX_E4M3, true>), g, b, 0, st, a);
    else hipLaunchKernelGGL((mx_dequant_kernel<MOE_MX_E4M3, false>), g, b, 0, st, a);
    return check_launch("mx_dequant");
}

extern "C" int mx_add_norm_quant(const uint16_t* x, int64_t x_row_stride, const uint16_t* residual,
                                 int64_t residual_row_stride, const uint16_t* norm_weight, float gain_center,
                                 float eps, int T, int H, int fmt, uint16_t* sum, int64_t sum_row_stride,
                                 uint8_t* codes, uint8_t* sf, void* stream) {
    using namespace moe;
    const char* name = "mx_add_norm_quant";
    const int rc = mx_check(x, x_row_stride, T, H, fmt, codes, sf, name);
    if (rc != MOE_OK) return rc;
    if (H > MOE_MAX_HIDDEN) return fail(MOE_EUNSUPPORTED, "%s: H=%d above %d", name, H, MOE_MAX_HIDDEN);
    if (!launch_fits(T, 1024)) return fail(MOE_EUNSUPPORTED, "%s: too many rows", name);
    if (!(eps > 0.0f) || eps > 1.0f || !(gain_center == gain_center))
        return fail(MOE_EINVAL, "%s: eps must be in (0, 1] and the gain centre a number", name);
    if (T == 0 || H == 0) return MOE_OK;
    if (residual && !sum) return fail(MOE_EINVAL, "%s: a residual needs the buffer of the sum", name);
    if ((residual && !aligned16(residual)) || (sum && !aligned16(sum)) || (norm_weight && !aligned16(norm_weight)))
        return fail(MOE_EINVAL, "%s: pointers must be 16-byte aligned", name);
    if ((residual && (residual_row_stride < H || residual_row_stride % 8)) ||
        (sum && (sum_row_stride < H || sum_row_stride % 8)))
        return fail(MOE_EINVAL, "%s: row strides must be >= H and multiples of 8", name);
    if (sum && ((sum == residual && sum_row_stride != residual_row_stride) ||
                (sum == x && sum_row_stride != x_row_stride)))
        return fail(MOE_EINVAL, "%s: a sum in place of an input needs its row stride", name);
    AnArgs a{x, x_row_stride, residual, residual_row_stride, norm_weight, gain_center, eps, T, H, sum, sum_row_stride,
             codes, sf};
    if (fmt == MOE_MX_E2M1) launch_add_norm<MOE_MX_E2M1>(a, (hipStream_t)stream);
    else launch_add_norm<MOE_MX_E4M3>(a, (hipStream_t)stream);
    return check_launch(name);
}
