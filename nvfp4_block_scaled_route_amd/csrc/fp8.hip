// Dense products of e4m3 operands with one fp32 scale for each block of 128, and
// their quantizers:
//   fp8_quant         x -> codes, a scale for each 1 x 128
//   fp8_quant_weight  w -> codes, a scale for each 128 x 128, and both transposed
//   fp8_gemm          out[t, n] = sum_b a_sf[b, t] w_sf[n/128, b] sum_{k in b} a[t, k] w[n, k]
#include "experts.hpp"
#include "mx.hpp"

namespace moe {

constexpr int kFpBlock = 128;
constexpr float kFpLeast = 7.888609052210118e-31f;      // 2^-100: the least maximum that a scale is made for

// The multipliers of a block from the bits of its largest magnitude m: q = 448 v / m
// as (0.875 v) / (m 2^-9), both sides exact, the division rounded once.
struct FpBlock {
    float d, r, sf;     // m 2^-9, its reciprocal, m / 448
    bool bad;           // an infinity or a NaN in the block
};
__device__ __forceinline__ FpBlock fp_block(uint32_t amax_bits) {
    FpBlock b;
    b.bad = amax_bits >= 0x7F800000u;
    const float m = fmaxf(__uint_as_float(amax_bits), kFpLeast);
    b.d = __fmul_rn(m, 0.001953125f);
    b.r = __fdiv_rn(1.0f, b.d);
    b.sf = b.bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(m, 448.0f);
    return b;
}

// The quotient from the reciprocal and one correction, the remainder exact (fused
// multiply-adds). e4m3's ties are 5-bit numbers, and v and m have 8 bits: a quotient
// is a tie, which the correction gives whole, or 2^-14 away from one.
__device__ __forceinline__ float fp_quot(float v, const FpBlock& b) {
    const float y = __fmul_rn(v, 0.875f), q = __fmul_rn(y, b.r);
    return __fmaf_rn(__fmaf_rn(-q, b.d, y), b.r, q);
}

__device__ __forceinline__ uint2 fp_codes8(const float (&v)[8], const FpBlock& b) {
    if (b.bad) return make_uint2(0u, 0u);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf(fp_quot(v[i], b), -448.0f), 448.0f);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// The maximum over a row of 16 lanes, in all of them.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    v = quad_max(v);
    const uint32_t a = (uint32_t)dpp_i<kDppRowHalfMirror>((int)v);
    v = v > a ? v : a;
    const uint32_t b = (uint32_t)dpp_i<kDppRowMirror>((int)v);
    return v > b ? v : b;
}

struct FqArgs {
    const uint16_t* x;
    int64_t x_row_stride;
    int T, H, blocks;
    uint8_t* codes;
    float* sf;
    int64_t sf_stride;
};

// A lane owns 8 values, 16 lanes a block; a workgroup 16 rows of one column of
// blocks, whose scales lie side by side.
__global__ void __launch_bounds__(256) fp8_quant_kernel(FqArgs a) {
    const int64_t rows = blockIdx.x / a.blocks;
    const int b = (int)(blockIdx.x - rows * a.blocks), lane16 = threadIdx.x & 15;
    const int64_t t = rows * 16 + (threadIdx.x >> 4);
    const int h = b * kFpBlock + lane16 * 8;
    float v[8];
    const bool live = t < a.T && h < a.H;
    unpack8(live ? *reinterpret_cast<const uint4*>(a.x + t * a.x_row_stride + h) : make_uint4(0u, 0u, 0u, 0u), v);
    const FpBlock s = fp_block(row16_max(amax8_bits(v)));
    if (live) *reinterpret_cast<uint2*>(a.codes + t * a.H + h) = fp_codes8(v, s);
    if (lane16 == 0 && t < a.T) a.sf[b * a.sf_stride + t] = s.sf;
}

struct FwArgs {
    const uint16_t* w;
    int64_t w_row_stride;
    int N, K;
    uint8_t* codes;
    float* sf;
    uint8_t* codes_t;       // or NULL
    int64_t codes_t_stride;
    float* sf_t;
};

// Byte i of 4 words -> word i, the words' bytes in order.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
    const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
    const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
    w[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
    w[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
    w[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
    w[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// A workgroup a block of 128 x 128, a thread 8 x 8 of it in registers from the
// load to the codes; the transposed ones go through LDS to whole rows.
__global__ void __launch_bounds__(256) fp8_quant_weight_kernel(FwArgs a) {
    constexpr int kRow = 128 + 16;
    __shared__ __align__(16) uint8_t s_t[128 * kRow];
    __shared__ uint32_t s_max[4];
    const int across = (a.K + 127) / 128, bn = blockIdx.x / across, bk = blockIdx.x - bn * across;
    const int tid = threadIdx.x, c = (tid & 15) * 8, r = (tid >> 4) * 8, n0 = bn * 128, k0 = bk * 128;
    float v[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool live = n0 + r + i < a.N && k0 + c < a.K;
        unpack8(live ? *reinterpret_cast<const uint4*>(a.w + (int64_t)(n0 + r + i) * a.w_row_stride + k0 + c) : make_uint4(0u, 0u, 0u, 0u),
                v[i]);
        const uint32_t mi = amax8_bits(v[i]);
        m = m > mi ? m : mi;
    }
    m = row16_max(m);
#pragma unroll
    for (int off = 16; off < 64; off <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)m, off);
        m = m > o ? m : o;
    }
    if ((tid & 63) == 0) s_max[tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) m = m > s_max[w] ? m : s_max[w];
    const FpBlock s = fp_block(m);
    uint2 code[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        code[i] = fp_codes8(v[i], s);
        if (n0 + r + i < a.N && k0 + c < a.K) *reinterpret_cast<uint2*>(a.codes + (int64_t)(n0 + r + i) * a.K + k0 + c) = code[i];
    }
    if (tid == 0) a.sf[blockIdx.x] = s.sf;
    if (!a.codes_t) return;
    if (tid == 0) a.sf_t[bk * ((a.N + 127) / 128) + bn] = s.sf;
    uint32_t q[2][2][4];        // rows' and columns' halves
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[0][0][i] = code[i].x, q[0][1][i] = code[i].y;
        q[1][0][i] = code[4 + i].x, q[1][1][i] = code[4 + i].y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) transpose4(q[i >> 1][i & 1]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint2*>(s_t + (c + j) * kRow + r) = make_uint2(q[0][j >> 2][j & 3], q[1][j >> 2][j & 3]);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = (tid >> 3) + 32 * j, n = (tid & 7) * 16;
        if (k0 + k >= a.K || n0 + n >= a.N) continue;
        const uint8_t* src = s_t + k * kRow + n;
        uint8_t* dst = a.codes_t + (k0 + k) * a.codes_t_stride + n0 + n;
        if (n0 + n + 16 <= a.N) {
            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
        } else {
            for (int i = 0; n0 + n + i < a.N; ++i) dst[i] = src[i];
        }
    }
}

// ------------------------------------------------------------------ product
typedef int fp_i8 __attribute__((ext_vector_type(8)));
typedef float fp_f16v __attribute__((ext_vector_type(16)));

struct FgArgs {
    const uint8_t* a;
    const float* a_sf;
    int64_t a_sf_stride;
    const uint8_t* w;
    int64_t w_row_stride;
    const float* w_sf;
    int T, N, K;
    uint16_t* out;
    int64_t out_stride;
    int out_vec;
};

// Direct-to-LDS load of one word a lane, as lds_copy16.
__device__ __forceinline__ void fp_copy4(u32x4 rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
    asm volatile("buffer_load_dword %0, %1, %2 offen lds" :: "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds) : "memory");
}

template <int WM, int WN, int MW, int NW>
struct FgShape {
    static constexpr int kWaves = WM * WN, kBM = 32 * WM * MW, kBN = 32 * WN * NW;
    static constexpr int kACopies = kBM * 128 / (1024 * kWaves), kWCopies = kBN * 128 / (1024 * kWaves), kAll = kACopies + kWCopies + 1;
    static constexpr int kSfBytes = kBM < 64 ? 256 : 4 * kBM;
    static constexpr int kW = kBM * 128, kSf = kW + kBN * 128, kStage = kSf + kSfBytes;
    static constexpr int kPerCu = kBM * kBN >= 256 * 256 ? 1 : 2;
    static constexpr int kFit = 160 * 1024 / kPerCu / kStage, kRing = kFit < 6 ? kFit : 6;
    static_assert(kRing >= 2 && (kRing - 1) * kAll < 64 && kACopies >= 1 && kWCopies >= 1, "ring of stages");
};

__device__ __forceinline__ int fp_swizzle(int chunk, int row) { return chunk ^ (row & 7) ^ ((row >> 3) & 1); }

// A stage is one block of K: 128 bytes of every row. The block's products are summed
// by the matrix cores from zero, and the sum is added to the accumulators under its
// scale, a's times w's: with the weights as the MFMA's rows a lane holds 16 columns
// of one token, all under one scale.
template <int WM, int WN, int MW, int NW>
__global__ void __launch_bounds__(64 * WM * WN, (FgShape<WM, WN, MW, NW>::kPerCu * WM * WN / 4)) fp8_gemm_kernel(FgArgs a) {
    using S = FgShape<WM, WN, MW, NW>;
    constexpr int kOutRow = 64 * NW + 16, kLds = S::kRing * S::kStage > S::kWaves * 32 * kOutRow ? S::kRing * S::kStage : S::kWaves * 32 * kOutRow;
    __shared__ __align__(16) uint8_t lds[kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, g = lane >> 5, wm = wave / WN, wn = wave % WN;
    const int mt = (a.T + S::kBM - 1) / S::kBM, nt = (a.N + S::kBN - 1) / S::kBN, tiles = mt * nt;
    const int x = blockIdx.x & 7, per = tiles >> 3, more = tiles & 7;
    const int id = x * per + (x < more ? x : more) + (int)(blockIdx.x >> 3);
    const int gm0 = id / (4 * nt) * 4, gh = mt - gm0 < 4 ? mt - gm0 : 4, in = id - gm0 * nt;
    const int m0 = (gm0 + in % gh) * S::kBM, n0 = (in / gh) * S::kBN;

    const int stages = (a.K + 127) / 128;
    const u32x4 ra = buffer_desc(a.a + (int64_t)m0 * a.K), rw = buffer_desc(a.w + n0 * a.w_row_stride), rs = buffer_desc(a.a_sf + m0);
    uint32_t offa[S::kACopies], offw[S::kWCopies], offs;
    const int r0 = 8 * wave + lane / 8, chunk = fp_swizzle(lane % 8, r0);
#pragma unroll
    for (int q = 0; q < S::kACopies; ++q) {
        const int row = r0 + 8 * S::kWaves * q;
        offa[q] = m0 + row < a.T ? (uint32_t)(row * a.K + chunk * 16) : 0x80000000u;
    }
#pragma unroll
    for (int q = 0; q < S::kWCopies; ++q) {
        const int row = r0 + 8 * S::kWaves * q;
        offw[q] = n0 + row < a.N ? (uint32_t)(row * a.w_row_stride + chunk * 16) : 0x80000000u;
    }
    const int part = wave % (S::kSfBytes / 256), srow = part * 64 + lane;
    offs = srow < S::kBM && m0 + srow < a.T ? (uint32_t)(4 * srow) : 0x80000000u;
    const uint32_t lds0 = lds_addr(lds);
    auto copy = [&](int s, int q0, int q1) {
        const uint32_t at = lds0 + (s % S::kRing) * S::kStage;
        const bool in_k = s * 128 + chunk * 16 < a.K;
#pragma unroll
        for (int q = q0; q < q1; ++q) {
            if (q < S::kACopies)
                lds_copy16(ra, __builtin_amdgcn_readfirstlane(at + (S::kWaves * q + wave) * 1024), in_k ? offa[q] : 0x80000000u, s * 128);
            else if (q < S::kACopies + S::kWCopies)
                lds_copy16(rw, __builtin_amdgcn_readfirstlane(at + S::kW + (S::kWaves * (q - S::kACopies) + wave) * 1024),
                           in_k ? offw[q - S::kACopies] : 0x80000000u, s * 128);
            else        // the stage's scales; waves repeat each other's
                fp_copy4(buffer_desc(a.a_sf + m0 + (s < stages ? s : 0) * a.a_sf_stride),
                         __builtin_amdgcn_readfirstlane(at + S::kSf + part * 256), offs, 0u);
        }
    };
    struct Frag {
        uint4 q[2];
        __device__ __forceinline__ fp_i8 reg() const {
            return fp_i8{(int)q[0].x, (int)q[0].y, (int)q[0].z, (int)q[0].w, (int)q[1].x, (int)q[1].y, (int)q[1].z, (int)q[1].w};
        }
    };
    auto read = [&](const uint8_t* rows, int row, Frag (&f)[2]) {
        const uint8_t* p = rows + row * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) f[h].q[i] = *reinterpret_cast<const uint4*>(p + 16 * fp_swizzle(4 * h + 2 * i + g, row));
    };
    // this wave's columns lie in one block of w's scales; lane i holds that of stage 64 j + i
    const float* wsf = a.w_sf + (int64_t)((n0 + 32 * NW * wn) / 128) * stages;
    const bool cols = n0 + 32 * NW * wn < a.N;
    float sw64 = 0.0f;

    fp_f16v acc[MW][NW];
#pragma unroll
    for (int m = 0; m < MW; ++m)
#pragma unroll
        for (int n = 0; n < NW; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.0f;

#pragma unroll
    for (int s = 0; s < S::kRing; ++s) copy(s, 0, S::kAll);
    Frag fw[NW][2], fa[MW][2];
    float sa[MW];
    __builtin_amdgcn_s_waitcnt(vmcnt_at_most((S::kRing - 1) * S::kAll));
    __syncthreads();
    for (int s = 0; s < stages; ++s) {
        const uint8_t* at = lds + (s % S::kRing) * S::kStage;
        if ((s & 63) == 0) sw64 = cols && s + lane < stages ? wsf[s + lane] : 0.0f;
#pragma unroll
        for (int n = 0; n < NW; ++n) read(at + S::kW, 32 * (wn * NW + n) + r, fw[n]);
#pragma unroll
        for (int m = 0; m < MW; ++m) {
            read(at, 32 * (wm * MW + m) + r, fa[m]);
            sa[m] = *reinterpret_cast<const float*>(at + S::kSf + 4 * (32 * (wm * MW + m) + r));
        }
        const float sw = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sw64), s & 63));
#pragma unroll
        for (int m = 0; m < MW; ++m) {
            if (m == MW - 1) {
                __builtin_amdgcn_s_waitcnt(vmcnt_at_most((S::kRing - 2) * S::kAll) & lgkmcnt_zero());
                asm volatile("s_barrier" ::: "memory");
                copy(s + S::kRing, 0, S::kAll);
            }
            const float f = __fmul_rn(sa[m], sw);
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                fp_f16v t = {};
                t = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[n][0].reg(), fa[m][0].reg(), t, 0, 0, 0, 0, 0, 0);
                t = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[n][1].reg(), fa[m][1].reg(), t, 0, 0, 0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[m][n][i] = __fmaf_rn(f, t[i], acc[m][n][i]);
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_at_most(0) & lgkmcnt_zero());
    __syncthreads();

    uint8_t* slab = lds + wave * 32 * kOutRow;
#pragma unroll
    for (int m = 0; m < MW; ++m) {
        wave_lds_sync();
#pragma unroll
        for (int n = 0; n < NW; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint2*>(slab + r * kOutRow + 2 * (32 * n + 8 * q + 4 * g)) =
                    make_uint2(f32_to_bf16(acc[m][n][4 * q]) | (f32_to_bf16(acc[m][n][4 * q + 1]) << 16),
                               f32_to_bf16(acc[m][n][4 * q + 2]) | (f32_to_bf16(acc[m][n][4 * q + 3]) << 16));
        wave_lds_sync();
        const int t0 = m0 + 32 * (wm * MW + m), c0 = n0 + 32 * NW * wn;
#pragma unroll
        for (int j = 0; j < 2 * NW; ++j) {
            const int i = lane + 64 * j, row = i / (4 * NW), c = i % (4 * NW) * 8;
            if (t0 + row >= a.T || c0 + c >= a.N) continue;
            uint16_t* dst = a.out + (t0 + row) * a.out_stride + c0 + c;
            const uint16_t* src = reinterpret_cast<const uint16_t*>(slab + row * kOutRow + 2 * c);
            if (a.out_vec && c0 + c + 8 <= a.N) {
                *reinterpret_cast<u32x4*>(dst) = *reinterpret_cast<const u32x4*>(src);
            } else {
                for (int k = 0; k < 8 && c0 + c + k < a.N; ++k) dst[k] = src[k];
            }
        }
    }
}

template <int WM, int WN, int MW, int NW>
int launch_fp8(const FgArgs& a, hipStream_t s) {
    using S = FgShape<WM, WN, MW, NW>;
    const int64_t tiles = (int64_t)((a.T + S::kBM - 1) / S::kBM) * ((a.N + S::kBN - 1) / S::kBN);
    if (!launch_fits(tiles, 64 * S::kWaves)) return fail(MOE_EUNSUPPORTED, "fp8_gemm: too many output tiles");
    hipLaunchKernelGGL((fp8_gemm_kernel<WM, WN, MW, NW>), dim3((unsigned)tiles), dim3(64 * S::kWaves), 0, s, a);
    return check_launch("fp8_gemm");
}

}  // namespace moe

extern "C" int fp8_quant(const uint16_t* x, int64_t x_row_stride, int T, int H, uint8_t* codes, float* sf, int64_t sf_stride,
                         void* stream) {
    using namespace moe;
    const char* name = "fp8_quant";
    if (T < 0 || H < 0) return fail(MOE_EINVAL, "%s: negative size T=%d H=%d", name, T, H);
    if (H % 16) return fail(MOE_EUNSUPPORTED, "%s: H=%d is not a multiple of 16", name, H);
    if (T == 0 || H == 0) return MOE_OK;
    if (!x || !codes || !sf) return fail(MOE_EINVAL, "%s: NULL pointer", name);
    if (!aligned16(x) || !aligned16(codes) || !aligned16(sf)) return fail(MOE_EINVAL, "%s: pointers must be 16-byte aligned", name);
    if (x_row_stride < H || x_row_stride % 8)
        return fail(MOE_EINVAL, "%s: row stride %lld must be >= H and a multiple of 8", name, (long long)x_row_stride);
    if (sf_stride < T) return fail(MOE_EINVAL, "%s: scale stride %lld must be >= T", name, (long long)sf_stride);
    FqArgs a{x, x_row_stride, T, H, (H + 127) / 128, codes, sf, sf_stride};
    const int64_t grid = (int64_t)((T + 15) / 16) * a.blocks;
    if (!launch_fits(grid, 256)) return fail(MOE_EUNSUPPORTED, "%s: too large", name);
    hipLaunchKernelGGL(fp8_quant_kernel, dim3((unsigned)grid), dim3(256), 0, (hipStream_t)stream, a);
    return check_launch(name);
}

extern "C" int fp8_quant_weight(const uint16_t* w, int64_t w_row_stride, int N, int K, uint8_t* codes, float* sf, uint8_t* codes_t,
                                int64_t codes_t_stride, float* sf_t, void* stream) {
    using namespace moe;
    const char* name = "fp8_quant_weight";
    if (N < 0 || K < 0) return fail(MOE_EINVAL, "%s: negative size N=%d K=%d", name, N, K);
    if (K % 16) return fail(MOE_EUNSUPPORTED, "%s: K=%d is not a multiple of 16", name, K);
    if (N == 0 || K == 0) return MOE_OK;
    if (!w || !codes || !sf) return fail(MOE_EINVAL, "%s: NULL pointer", name);
    if (!codes_t != !sf_t) return fail(MOE_EINVAL, "%s: transposed codes and scales go together", name);
    if (!aligned16(w) || !aligned16(codes) || !aligned16(sf) || !aligned16(codes_t) || !aligned16(sf_t))
        return fail(MOE_EINVAL, "%s: pointers must be 16-byte aligned", name);
    if (w_row_stride < K || w_row_stride % 8)
        return fail(MOE_EINVAL, "%s: row stride %lld must be >= K and a multiple of 8", name, (long long)w_row_stride);
    if (codes_t && (codes_t_stride < N || codes_t_stride % 16))
        return fail(MOE_EINVAL, "%s: transposed row stride %lld must be >= N and a multiple of 16", name, (long long)codes_t_stride);
    FwArgs a{w, w_row_stride, N, K, codes, sf, codes_t, codes_t_stride, sf_t};
    const int64_t grid = (int64_t)((N + 127) / 128) * ((K + 127) / 128);
    if (!launch_fits(grid, 256)) return fail(MOE_EUNSUPPORTED, "%s: too large", name);
    hipLaunchKernelGGL(fp8_quant_weight_kernel, dim3((unsigned)grid), dim3(256), 0, (hipStream_t)stream, a);
    return check_launch(name);
}

extern "C" int fp8_gemm(const uint8_t* a_codes, const float* a_sf, int64_t a_sf_stride, const uint8_t* w_codes, int64_t w_row_stride,
                        const float* w_sf, int T, int N, int K, uint16_t* out, int64_t out_row_stride, void* stream) {
    using namespace moe;
    const char* name = "fp8_gemm";
    if (T < 0 || N < 0 || K < 0) return fail(MOE_EINVAL, "%s: negative size T=%d N=%d K=%d", name, T, N, K);
    if (K < 16 || K % 16 || K > MOE_MAX_MX_K)
        return fail(MOE_EUNSUPPORTED, "%s: K=%d must be a multiple of 16 in [16, %d]", name, K, MOE_MAX_MX_K);
    if (T == 0 || N == 0) return MOE_OK;
    if (!a_codes || !a_sf || !w_codes || !w_sf || !out) return fail(MOE_EINVAL, "%s: NULL pointer", name);
    if (!aligned16(a_codes) || !aligned16(a_sf) || !aligned16(w_codes) || !aligned16(w_sf) || !aligned16(out))
        return fail(MOE_EINVAL, "%s: pointers must be 16-byte aligned", name);
    if (a_sf_stride < T) return fail(MOE_EINVAL, "%s: scale stride %lld must be >= T", name, (long long)a_sf_stride);
    if (w_row_stride < K || w_row_stride % 16 || w_row_stride > (1 << 22))
        return fail(MOE_EINVAL, "%s: weight row stride %lld must be >= K, a multiple of 16 and at most %d", name, (long long)w_row_stride,
                    1 << 22);
    if (out_row_stride < N) return fail(MOE_EINVAL, "%s: out row stride %lld must be >= N", name, (long long)out_row_stride);
    FgArgs a{a_codes, a_sf, a_sf_stride, w_codes, w_row_stride, w_sf, T, N, K, out, out_row_stride, out_row_stride % 8 == 0 ? 1 : 0};
    hipStream_t s = (hipStream_t)stream;
    if (T <= 64) return launch_fp8<1, 4, 1, 1>(a, s);
    if ((int64_t)T * N >= 2048 * 2048) return launch_fp8<2, 4, 4, 2>(a, s);
    return launch_fp8<2, 2, 2, 2>(a, s);
}
