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
// is a tie, which the correction gives whole, or 2^-14 away from one. (It loses a
// zero's sign: that is v's.)
__device__ __forceinline__ float fp_quot(float v, const FpBlock& b) {
    const float y = __fmul_rn(v, 0.875f), q = __fmul_rn(y, b.r);
    return __builtin_copysignf(__fmaf_rn(__fmaf_rn(-q, b.d, y), b.r, q), v);
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

// Sizes behind whose last row or column a block of 256 stays in 31 bits.
static int fp_sizes(int rows, int cols, const char* name) {
    return rows <= MOE_MAX_ROWS && cols <= MOE_MAX_ROWS ? MOE_OK
                                                        : fail(MOE_EUNSUPPORTED, "%s: %d x %d: a side is more than %d", name, rows, cols, MOE_MAX_ROWS);
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
// blocks, whose scales lie side by side. HBM-bound: 4096 x 4096 in 10.6 to 11.2 us,
// 4.5 to 4.8 TB/s, as a large copy.
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
// load to the codes; the transposed ones go through LDS to whole rows. HBM-bound:
// 4096 x 4096 with both outputs in 14.1 to 15.3 us, 4.4 to 4.8 TB/s.
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
// A block of K is one 16 x 16 x 128 MFMA, from zero; its sum is added to the
// accumulators under its scale, a's times w's, in fp32. Inside the block the matrix unit
// cuts each product to 13 bits below the largest of its 8, 1.5e-5 of a result: 2% of the
// bf16 outputs are the neighbours of the exact result's rounding (0.07% with sums in
// fp32), and the error of all against 64 bits is that rounding's, 1.662e-3 of the norm
// for 1.661e-3. Exact products would need bf16 operands, at half the matrix unit's rate.
// With the weights as the MFMA's rows a lane holds 4 columns of one token (lane & 15),
// all under one scale.
// A lane's operand is 16 bytes at element 16 g and 16 at 64 + 16 g, g = lane / 16.
typedef int fp_i8 __attribute__((ext_vector_type(8)));

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

struct FpFrag {
    uint4 q[2];
    __device__ __forceinline__ fp_i8 reg() const {
        return fp_i8{(int)q[0].x, (int)q[0].y, (int)q[0].z, (int)q[0].w, (int)q[1].x, (int)q[1].y, (int)q[1].z, (int)q[1].w};
    }
};

__device__ __forceinline__ floatx4 fp_mfma(const FpFrag& w, const FpFrag& a) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.reg(), a.reg(), floatx4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

// ------------------------------------------------------------------ few tokens
// A stream of the weights: a workgroup owns 16 columns, its 8 waves split the blocks
// of K, and the waves' sums are added through LDS in wave order. One token x 4096 x
// 4096 in 5.1 us, of which 2.4 are a launch's: bound by the time that the loads of a
// wave's 4 blocks, issued together, take to arrive.
constexpr int kFsWaves = 8;

template <int TM>
__global__ void __launch_bounds__(64 * kFsWaves) fp8_gemm_skinny_kernel(FgArgs a) {
    constexpr int U = 4;            // blocks whose loads issue together
    __shared__ floatx4 s_sum[kFsWaves][TM][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16, blocks = (a.K + 127) / 128;
    const uint8_t* wrow = a.w + (n0 + r < a.N ? n0 + r : a.N - 1) * a.w_row_stride + 16 * g;
    const uint8_t* arow[TM];
    const float* asf[TM];
#pragma unroll
    for (int m = 0; m < TM; ++m) {
        const int t = 16 * m + r < a.T ? 16 * m + r : a.T - 1;
        arow[m] = a.a + (int64_t)t * a.K + 16 * g;
        asf[m] = a.a_sf + t;
    }
    const float* wsf = a.w_sf + (int64_t)(n0 / 128) * blocks;       // 16 columns lie in one block
    floatx4 acc[TM];
#pragma unroll
    for (int m = 0; m < TM; ++m) acc[m] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    const int per = (blocks + kFsWaves - 1) / kFsWaves, b0 = wave * per, b1 = b0 + per < blocks ? b0 + per : blocks;
    for (int b = b0; b < b1; b += U) {
        FpFrag fw[U], fa[U][TM];
        float sa[U][TM], sw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int left = b + u < b1 ? a.K - 128 * (b + u) - 16 * g : 0;     // bytes of K from this lane's on
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t at = 128 * (int64_t)(b + u) + 64 * h;
                fw[u].q[h] = left > 64 * h ? *reinterpret_cast<const uint4*>(wrow + at) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int m = 0; m < TM; ++m)
                    fa[u][m].q[h] = left > 64 * h ? *reinterpret_cast<const uint4*>(arow[m] + at) : make_uint4(0u, 0u, 0u, 0u);
            }
            sw[u] = b + u < b1 ? wsf[b + u] : 0.0f;
#pragma unroll
            for (int m = 0; m < TM; ++m) sa[u][m] = b + u < b1 ? asf[m][(b + u) * a.a_sf_stride] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const float f = __fmul_rn(sa[u][m], sw[u]);
                const floatx4 t = fp_mfma(fw[u], fa[u][m]);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][i] = __fmaf_rn(f, t[i], acc[m][i]);
            }
    }
#pragma unroll
    for (int m = 0; m < TM; ++m) s_sum[wave][m][lane] = acc[m];
    __syncthreads();
    if (wave >= TM) return;
    floatx4 sum = s_sum[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kFsWaves; ++w) sum += s_sum[w][wave][lane];
    const int t = 16 * wave + r, n = n0 + 4 * g;
    if (t >= a.T) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < a.N) a.out[t * a.out_stride + n + i] = (uint16_t)f32_to_bf16(sum[i]);
}

// ------------------------------------------------------------------ many tokens
// Direct-to-LDS load of one word a lane, as lds_copy16.
__device__ __forceinline__ void fp_copy4(u32x4 rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
    asm volatile("buffer_load_dword %0, %1, %2 offen lds" :: "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds) : "memory");
}

// *p, or 0, waited for here: a wait at the use, which the compiler would put into
// every stage, would wait for the copies issued since too.
__device__ __forceinline__ float fp_load_wait(const float* p, bool on) {
    float v = on ? *p : 0.0f;
    asm volatile("" : "+v"(v));
    return v;
}

// LDS rows of NB blocks (128 or 256 bytes): the 16-byte chunks of a row permuted so
// that 16 consecutive rows' reads of one chunk spread over all banks.
template <int NB>
__device__ __forceinline__ int fp_swizzle(int chunk, int row) {
    return NB == 2 ? chunk ^ (row & 15) : chunk ^ (row & 7) ^ ((row >> 3) & 1);
}

// One workgroup's block of the output. Blocks of the output to workgroups: each XCD
// (workgroups are dealt to the 8 round robin) gets a contiguous run of them, which
// goes through groups of 4 rows of blocks column by column.
__device__ __forceinline__ void fp_block_of(int T, int N, int bm, int bn, int& m0, int& n0) {
    const int mt = (T + bm - 1) / bm, nt = (N + bn - 1) / bn, tiles = mt * nt;
    const int x = blockIdx.x & 7, per = tiles >> 3, more = tiles & 7;
    const int id = x * per + (x < more ? x : more) + (int)(blockIdx.x >> 3);
    const int gm0 = id / (4 * nt) * 4, gh = mt - gm0 < 4 ? mt - gm0 : 4, in = id - gm0 * nt;
    m0 = (gm0 + in % gh) * bm, n0 = (in / gh) * bn;
}

// 16 tokens of a wave's 16 NW columns, turned in the wave's own part of the LDS to
// whole pieces of their rows.
template <int NW>
__device__ __forceinline__ void fp_store(const FgArgs& a, uint8_t* slab, const floatx4 (&acc)[NW], int t0, int c0, int lane) {
    constexpr int kOutRow = 32 * NW + 16;
    const int r = lane & 15, g = lane >> 4;
    wave_lds_sync();
#pragma unroll
    for (int n = 0; n < NW; ++n)
        *reinterpret_cast<uint2*>(slab + r * kOutRow + 2 * (16 * n + 4 * g)) =
            make_uint2(bf16x2_pack(acc[n][0], acc[n][1]), bf16x2_pack(acc[n][2], acc[n][3]));
    wave_lds_sync();
    if (a.out_vec && a.N % 8 == 0) {
#pragma unroll
        for (int j = 0; j < (NW + 1) / 2; ++j) {        // 2 NW pieces of 16 bytes a row
            const int i = lane + 64 * j, row = i / (2 * NW), c = i % (2 * NW) * 8;
            if (row >= 16 || t0 + row >= a.T || c0 + c >= a.N) continue;
            __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(slab + row * kOutRow + 2 * c),
                                        reinterpret_cast<u32x4*>(a.out + (t0 + row) * a.out_stride + c0 + c));
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 4 * NW; ++j) {                  // a row's values by consecutive lanes
        const int i = lane + 64 * j, row = i / (16 * NW), c = i % (16 * NW);
        if (t0 + row < a.T && c0 + c < a.N)
            a.out[(t0 + row) * a.out_stride + c0 + c] = *reinterpret_cast<const uint16_t*>(slab + row * kOutRow + 2 * c);
    }
}

// 4 waves, 2 x 2, each MW x NW tiles of 16 x 16; a stage is NB blocks of K. KS such
// groups of waves with a ring each take turns at the stages.
template <int MW, int NW, int NB, int KS>
struct FgShape {
    static constexpr int kBM = 32 * MW, kBN = 32 * NW, kRow = 128 * NB;
    static constexpr int kACopies = kBM * kRow / 4096, kWCopies = kBN * kRow / 4096, kAll = kACopies + kWCopies + 1;
    static constexpr int kParts = kBM / 64;             // of 64 tokens' scales
    static constexpr int kW = kBM * kRow, kSf = kW + kBN * kRow, kStage = kSf + NB * 4 * kBM;
    static constexpr int kFit = 80 * 1024 / kStage, kRing = kFit < 4 ? kFit : 4;
    static constexpr int kSlab = 16 * (32 * NW + 16), kGroup = kRing * kStage, kLds = KS * kGroup;
    static_assert(4 * KS * kSlab <= kGroup && 4096 * MW * NW <= kGroup, "the waves' slabs and sums");
    static_assert(kRing >= 2 && kRing * kAll < 64 && kBM % 64 == 0 && kParts * NB <= 4 && 128 % (16 * NW) == 0, "ring of stages");
};

// The operands of a turn are read from LDS into registers while the products of the
// turn before run, so its buffer is free a turn early, and one barrier a turn does.
// A wave alone on its SIMD waits for each instruction it issues: copies, reads and
// sums are spread between the MFMAs (512 x 4096 x 4096 64 x 128 20.3 -> 15.5 us), and
// where the blocks are fewer than the CUs a second group of waves takes half of K
// (256 x 4096 x 4096 13.2 -> 10.9 us). 512 x 4096 x 4096 in 14.9 us: 1.15 PFLOP/s; rows
// that start inside a cache line cost their copies twice the lines (517 x 2088, K =
// 4096 13.9 us, K = 4112 18.1).
template <int MW, int NW, int NB, int KS>
__global__ void __launch_bounds__(256 * KS, 2) fp8_gemm_kernel(FgArgs a) {
    using S = FgShape<MW, NW, NB, KS>;
    __shared__ __align__(16) uint8_t all[S::kLds];
    const int lane = threadIdx.x & 63, w8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), group = w8 >> 2, wave = w8 & 3;
    uint8_t* lds = all + group * S::kGroup;
    const int r = lane & 15, g = lane >> 4, wm = wave >> 1, wn = wave & 1;
    int m0, n0;
    fp_block_of(a.T, a.N, S::kBM, S::kBN, m0, n0);

    const int blocks = (a.K + 127) / 128, stages = (blocks + NB - 1) / NB;
    const u32x4 ra = scalar_desc(a.a + (int64_t)m0 * a.K), rw = scalar_desc(a.w + n0 * a.w_row_stride);
    constexpr int kRowsPer = 8 / NB;        // rows that an instruction copies
    const int r0 = kRowsPer * wave + lane / (8 * NB), chunk = fp_swizzle<NB>(lane % (8 * NB), r0);      // rows 4 kRowsPer apart have the same
    const uint32_t offa = (uint32_t)(r0 * a.K + chunk * 16), offw = (uint32_t)(r0 * a.w_row_stride + chunk * 16);
    const int rows_a = a.T - m0 - r0, rows_w = a.N - n0 - r0;
    const int piece = wave % (S::kParts * NB), sblock = piece / S::kParts, stok = piece % S::kParts * 64 + lane;
    const uint32_t offs = m0 + stok < a.T ? (uint32_t)(4 * stok) : 0x80000000u;
    const uint32_t lds0 = lds_addr(lds);
    // copy q of the group's turn i (stage KS i + group): tokens', weights', scales'
    auto copy = [&](int i, int q) __attribute__((always_inline)) {
        const uint32_t at = lds0 + (i % S::kRing) * S::kStage;
        const int s = KS * i + group;
        const bool in_k = s * S::kRow + chunk * 16 < a.K;
        if (q < S::kACopies) {
            lds_copy16(ra, __builtin_amdgcn_readfirstlane(at + (4 * q + wave) * 1024),
                       in_k && 4 * kRowsPer * q < rows_a ? offa + (uint32_t)(4 * kRowsPer * q * a.K) : 0x80000000u, s * S::kRow);
        } else if (q < S::kAll - 1) {
            q -= S::kACopies;
            lds_copy16(rw, __builtin_amdgcn_readfirstlane(at + S::kW + (4 * q + wave) * 1024),
                       in_k && 4 * kRowsPer * q < rows_w ? offw + (uint32_t)(4 * kRowsPer * q * a.w_row_stride) : 0x80000000u, s * S::kRow);
        } else {
            const int b = s * NB + sblock;      // waves may repeat each other's
            fp_copy4(scalar_desc(a.a_sf + m0 + (b < blocks ? b : 0) * a.a_sf_stride), __builtin_amdgcn_readfirstlane(at + S::kSf + piece * 256),
                     b < blocks ? offs : 0x80000000u, 0u);
        }
    };
    struct Operands {
        FpFrag w[NB][NW], a[NB][MW];
        float sa[NB][MW];
    };
    // Read i of a turn's kReads: of each block the weights, then the tokens with their scale.
    constexpr int kReads = NB * (NW + MW);
    auto read = [&](int s, Operands& o, int i) __attribute__((always_inline)) {
        const uint8_t* at = lds + (s % S::kRing) * S::kStage;
        const int b = i / (NW + MW), j = i % (NW + MW);
        auto frag = [&](const uint8_t* rows, int row) __attribute__((always_inline)) {
            FpFrag f;
            f.q[0] = *reinterpret_cast<const uint4*>(rows + row * S::kRow + 16 * fp_swizzle<NB>(8 * b + g, row));
            f.q[1] = *reinterpret_cast<const uint4*>(rows + row * S::kRow + 16 * fp_swizzle<NB>(8 * b + 4 + g, row));
            return f;
        };
        if (j < NW) {
            o.w[b][j] = frag(at + S::kW, 16 * (wn * NW + j) + r);
        } else {
            const int row = 16 * (wm * MW + j - NW) + r;
            o.a[b][j - NW] = frag(at, row);
            o.sa[b][j - NW] = *reinterpret_cast<const float*>(at + S::kSf + 4 * (b * S::kBM + row));
        }
    };
    // this wave's columns lie in one block of w's scales; lane i holds that of block 64 j + i
    const float* wsf = a.w_sf + (int64_t)((n0 + 16 * NW * wn) / 128) * blocks;
    const bool cols = n0 + 16 * NW * wn < a.N;
    float sw64 = 0.0f;
    floatx4 acc[MW][NW];
#pragma unroll
    for (int m = 0; m < MW; ++m)
#pragma unroll
        for (int n = 0; n < NW; ++n) acc[m][n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    auto stage = [&](int s, const Operands& o, Operands& next) __attribute__((always_inline)) {
        __builtin_amdgcn_s_waitcnt(vmcnt_at_most((S::kRing - 2) * S::kAll) & lgkmcnt_zero());
        asm volatile("s_barrier" ::: "memory");
        // between the products: the copies of turn s + kRing, the reads of turn s + 1, the sums two products ago
        constexpr int kSlots = NB * MW * NW;
        floatx4 t[3];
        float f = 0.0f, last = 0.0f;
#pragma unroll
        for (int i = 0; i < kSlots + 2; ++i) {
            const int b = i / (MW * NW), m = i / NW % MW, n = i % NW;
            if (i < kSlots) {
                if (n == 0) {
                    last = f;
                    f = __fmul_rn(o.sa[b][m], __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sw64), ((KS * s + group) * NB + b) & 63)));
                }
                t[i % 3] = fp_mfma(o.w[b][n], o.a[b][m]);
#pragma unroll
                for (int q = i * S::kAll / kSlots; q < (i + 1) * S::kAll / kSlots; ++q) copy(s + S::kRing, q);
#pragma unroll
                for (int q = i * kReads / kSlots; q < (i + 1) * kReads / kSlots; ++q) read(s + 1, next, q);
            }
            if (i >= 2) {
                const int p = i - 2;
                const float scale = i >= kSlots || p / NW == i / NW ? f : last;
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[p / NW % MW][p % NW][k] = __fmaf_rn(scale, t[p % 3][k], acc[p / NW % MW][p % NW][k]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    static_assert(64 % (2 * KS * NB) == 0, "a pair of turns lies in 64 blocks");
#pragma unroll
    for (int s = 0; s < S::kRing; ++s)
#pragma unroll
        for (int q = 0; q < S::kAll; ++q) copy(s, q);
    Operands o0, o1;
    __builtin_amdgcn_s_waitcnt(vmcnt_at_most((S::kRing - 1) * S::kAll));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kReads; ++i) read(0, o0, i);
    const int turns = (stages + KS - 1) / KS;       // of either group: stages behind the last are zeros
    for (int s = 0; s < turns; s += 2) {
        if ((s * KS * NB & 63) == 0) sw64 = fp_load_wait(wsf + s * KS * NB + lane, cols && s * KS * NB + lane < blocks);
        stage(s, o0, o1);
        if (s + 1 < turns) stage(s + 1, o1, o0);
    }
    // the copies of the turns behind the last still write to the LDS
    __builtin_amdgcn_s_waitcnt(vmcnt_at_most(0) & lgkmcnt_zero());
    __syncthreads();
    // of two groups' sums each group stores half: the other's comes through LDS
    constexpr int kMine = MW / KS;
    if constexpr (KS == 2) {
        floatx4* sums = reinterpret_cast<floatx4*>(all) + (wave * MW * NW) * 64 + lane;
        static_assert(MW % 2 == 0, "halves");
#pragma unroll
        for (int m = 0; m < MW; ++m)
            if (m / kMine != group) {
#pragma unroll
                for (int n = 0; n < NW; ++n) sums[64 * (m * NW + n)] = acc[m][n];
            }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MW; ++m)
            if (m / kMine == group) {
#pragma unroll
                for (int n = 0; n < NW; ++n) acc[m][n] += sums[64 * (m * NW + n)];
            }
    }
    uint8_t* slab = KS == 2 ? all + S::kGroup + (4 * group + wave) * S::kSlab : all + wave * S::kSlab;      // clear of the sums
#pragma unroll
    for (int m = 0; m < MW; ++m) {
        const int t0 = m0 + 16 * (wm * MW + m);
        if (m / kMine == group && t0 < a.T && cols) fp_store<NW>(a, slab, acc[m], t0, n0 + 16 * NW * wn, lane);
    }
}

// 256 x 256: 8 waves, 2 x 4, of 128 x 64, which leaves a wave no registers to read
// a stage's operands beside the products of the one before; so the waves take
// turns: while 4 read, the other 4, one on each SIMD with them, multiply. Half steps
// end in barriers. Waves 0 to 3 read stage s in half step 2 s (the weights and their
// first 4 tiles of tokens; the other 4 while they multiply) and multiply in 2 s + 1,
// waves 4 to 7 one half step later. So stage s + 2 may be copied into s's buffer
// from half step 2 s + 2 on, but for the rows of the other tiles, which are read
// until its end, and come in 2 s + 3: the waves that read issue the copies, waves 0
// to 3 the first part and the others the second, and either has two half steps to
// arrive. The tokens' scales have 4 buffers.
//
// A SIMD's MFMA takes 32 cycles. A wave that has the matrix unit to itself, as the
// turns have it, issues one with the 4 additions of its sum in 41 (two waves at once take
// 35 each, as one's additions run beside the other's MFMA): 84 thousand of the 122
// thousand cycles that a CU is busy with 4096^3. The rest are its first stage, the ends
// of 64 half steps and the output.
struct FgWide {
    static constexpr int kSide = 256, kW = 256 * 128, kStage = 2 * 256 * 128, kSf = 2 * kStage, kLds = kSf + 4 * 1024;
};

__global__ void __launch_bounds__(512, 2) fp8_gemm_wide_kernel(FgArgs a) {
    using S = FgWide;
    __shared__ __align__(16) uint8_t lds[S::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4, wm = wave >> 2, wn = wave & 3;
    int m0, n0;
    fp_block_of(a.T, a.N, S::kSide, S::kSide, m0, n0);

    const int stages = (a.K + 127) / 128;
    const u32x4 ra = scalar_desc(a.a + (int64_t)m0 * a.K), rw = scalar_desc(a.w + n0 * a.w_row_stride);
    const int r0 = 8 * wn + lane / 8, chunk = fp_swizzle<1>(lane % 8, r0);          // rows 32 apart have the same
    const uint32_t lds0 = lds_addr(lds);
    const uint32_t offa = (uint32_t)(r0 * a.K + chunk * 16), offw = (uint32_t)(r0 * a.w_row_stride + chunk * 16);
    const int rows_a = a.T - m0 - r0, rows_w = a.N - n0 - r0;
    // Rows [32 q, 32 q + 32) of a stage, by the 4 waves of a group.
    auto copy_a = [&](int s, int q) __attribute__((always_inline)) {
        lds_copy16(ra, __builtin_amdgcn_readfirstlane(lds0 + (s & 1) * S::kStage + (4 * q + wn) * 1024),
                   s * 128 + chunk * 16 < a.K && 32 * q < rows_a ? offa + (uint32_t)(32 * q * a.K) : 0x80000000u, s * 128);
    };
    auto copy_first = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            lds_copy16(rw, __builtin_amdgcn_readfirstlane(lds0 + (s & 1) * S::kStage + S::kW + (4 * q + wn) * 1024),
                       s * 128 + chunk * 16 < a.K && 32 * q < rows_w ? offw + (uint32_t)(32 * q * a.w_row_stride) : 0x80000000u, s * 128);
        copy_a(s, 0);
        copy_a(s, 1);
        copy_a(s, 4);
        copy_a(s, 5);
        const int tok = wn * 64 + lane;
        fp_copy4(scalar_desc(a.a_sf + m0 + (s < stages ? s : 0) * a.a_sf_stride),
                 __builtin_amdgcn_readfirstlane(lds0 + S::kSf + (s & 3) * 1024 + wn * 256),
                 s < stages && m0 + tok < a.T ? (uint32_t)(4 * tok) : 0x80000000u, 0u);
    };
    auto copy_second = [&](int s) __attribute__((always_inline)) {
        copy_a(s, 2);
        copy_a(s, 3);
        copy_a(s, 6);
        copy_a(s, 7);
    };
    FpFrag fw[4], fa[5];        // tile m of the tokens in fa[m % 5]
    auto frag = [&](const uint8_t* rows, int row) __attribute__((always_inline)) {
        FpFrag f;
        f.q[0] = *reinterpret_cast<const uint4*>(rows + row * 128 + 16 * fp_swizzle<1>(g, row));
        f.q[1] = *reinterpret_cast<const uint4*>(rows + row * 128 + 16 * fp_swizzle<1>(4 + g, row));
        return f;
    };
    auto read = [&](int s) __attribute__((always_inline)) {
        const uint8_t* at = lds + (s & 1) * S::kStage;
#pragma unroll
        for (int n = 0; n < 4; ++n) fw[n] = frag(at + S::kW, 64 * wn + 16 * n + r);
#pragma unroll
        for (int m = 0; m < 4; ++m) fa[m] = frag(at, 128 * wm + 16 * m + r);
    };
    const float* wsf = a.w_sf + (int64_t)((n0 + 64 * wn) / 128) * stages;
    const bool cols = n0 + 64 * wn < a.N;
    float sw64 = 0.0f;
    floatx4 acc[8][4];
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) acc[m][n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    auto products = [&](int s) __attribute__((always_inline)) {
        const uint8_t* at = lds + (s & 1) * S::kStage;
        __builtin_amdgcn_s_setprio(1);
        const float sw = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sw64), s & 63));
        const uint8_t* sf = lds + S::kSf + (s & 3) * 1024 + 4 * (128 * wm + r);
        float f = 0.0f, last = 0.0f, sa = *reinterpret_cast<const float*>(sf);
        floatx4 t[4];
        // a sum is added two MFMAs after its own
#pragma unroll
        for (int i = 0; i < 34; ++i) {
            const int m = i / 4, n = i % 4;
            if (n == 0 && m < 8) {
                last = f;
                f = __fmul_rn(sa, sw);
                if (m < 7) sa = *reinterpret_cast<const float*>(sf + 64 * (m + 1));
                if (m < 4) fa[(m + 4) % 5] = frag(at, 128 * wm + 16 * (m + 4) + r);
            }
            if (i < 32) t[n] = fp_mfma(fw[n], fa[m % 5]);
            if (i >= 2) {
                const int pm = (i - 2) / 4, pn = (i - 2) % 4;
                const float scale = pm == m || i >= 32 ? f : last;
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[pm][pn][k] = __fmaf_rn(scale, t[pn][k], acc[pm][pn][k]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_setprio(0);
    };
    auto half = [&]() __attribute__((always_inline)) {       // the end of a half step
        __builtin_amdgcn_s_waitcnt(lgkmcnt_zero());
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto scales = [&](int s) __attribute__((always_inline)) {
        if ((s & 63) == 0) sw64 = fp_load_wait(wsf + s + lane, cols && s + lane < stages);
    };
    if (wm == 0) copy_first(0);
    else copy_second(0);
    __builtin_amdgcn_s_waitcnt(vmcnt_at_most(0));
    asm volatile("s_barrier" ::: "memory");
    if (wm == 0) {
        for (int s = 0; s < stages; ++s) {
            scales(s);
            copy_first(s + 1);                                  // half step 2 s
            read(s);
            half();
            products(s);                                        // 2 s + 1
            __builtin_amdgcn_s_waitcnt(vmcnt_at_most(0));
            half();
        }
        half();
    } else {
        half();                                                 // half step 0
        for (int s = 0; s < stages; ++s) {
            scales(s);
            copy_second(s + 1);                                 // 2 s + 1
            read(s);
            half();
            products(s);                                        // 2 s + 2
            __builtin_amdgcn_s_waitcnt(vmcnt_at_most(0));
            half();
        }
    }
    // the copies of the stages behind the last still write to the LDS
    __builtin_amdgcn_s_waitcnt(vmcnt_at_most(0) & lgkmcnt_zero());
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        const int t0 = m0 + 128 * wm + 16 * m;
        if (t0 < a.T && cols) fp_store<4>(a, lds + wave * 16 * (32 * 4 + 16), acc[m], t0, n0 + 64 * wn, lane);
    }
}

template <int MW, int NW, int NB, int KS>
int launch_fp8(const FgArgs& a, hipStream_t s) {
    using S = FgShape<MW, NW, NB, KS>;
    const int64_t tiles = (int64_t)((a.T + S::kBM - 1) / S::kBM) * ((a.N + S::kBN - 1) / S::kBN);
    if (!launch_fits(tiles, 256 * KS)) return fail(MOE_EUNSUPPORTED, "fp8_gemm: too many output tiles");
    hipLaunchKernelGGL((fp8_gemm_kernel<MW, NW, NB, KS>), dim3((unsigned)tiles), dim3(256 * KS), 0, s, a);
    return check_launch("fp8_gemm");
}

static int launch_fp8_wide(const FgArgs& a, hipStream_t s) {
    const int64_t tiles = (int64_t)((a.T + 255) / 256) * ((a.N + 255) / 256);
    if (!launch_fits(tiles, 512)) return fail(MOE_EUNSUPPORTED, "fp8_gemm: too many output tiles");
    hipLaunchKernelGGL(fp8_gemm_wide_kernel, dim3((unsigned)tiles), dim3(512), 0, s, a);
    return check_launch("fp8_gemm");
}

template <int TM>
int launch_fp8_skinny(const FgArgs& a, hipStream_t s) {
    const int64_t groups = ((int64_t)a.N + 15) / 16;
    hipLaunchKernelGGL(fp8_gemm_skinny_kernel<TM>, dim3((unsigned)groups), dim3(64 * kFsWaves), 0, s, a);
    return check_launch("fp8_gemm");
}

}  // namespace moe

extern "C" int fp8_quant(const uint16_t* x, int64_t x_row_stride, int T, int H, uint8_t* codes, float* sf, int64_t sf_stride,
                         void* stream) {
    using namespace moe;
    const char* name = "fp8_quant";
    if (T < 0 || H < 0) return fail(MOE_EINVAL, "%s: negative size T=%d H=%d", name, T, H);
    if (H % 16) return fail(MOE_EUNSUPPORTED, "%s: H=%d is not a multiple of 16", name, H);
    const int rc = fp_sizes(T, H, name);
    if (rc != MOE_OK || T == 0 || H == 0) return rc;
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
    const int rc = fp_sizes(N, K, name);
    if (rc != MOE_OK || N == 0 || K == 0) return rc;
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
    const int rc = fp_sizes(T, N, name);
    if (rc != MOE_OK || T == 0 || N == 0) return rc;
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
    // us, K = 4096, replayed from a graph: by columns, blocks of 64 x 64 with two groups of waves, of 64 x 128 with two
    // and with one, 128 x 128, 256 x 256
    //    1 x 4096   5.1 10.1 13.3 15.0 24.3 47     16 x 8192  10.4 10.1 13.0 14.8 24.3 48      1 x 16384 13.8 12.6 13.2 14.8 24.7 49
    //   32 x 4096   8.4 10.1 13.3 15.0 24.3 48    256 x 4096    -  10.9 13.8 15.4 25.2 49    512 x 4096    -  20.7 14.9 16.7 26.0 50
    //  768 x 4096    -  29.4 26.3 22.2 26.8 50   1024 x 4096    -  39.4 28.8 25.4 27.6 50   1280 x 4096    -  49.0 40.0 36.1 32.6 50
    // 2048 x 4096    -  74.9 55.9 49.7 38.8 52   3000 x 4096    -   111 83.8 72.9 60.9 55   8192 x 8192    -   555  421  362  287 245
    // 4096 x 4096    -   145  108 91.3 73.9 62   4096 x 4352    -   154  118 99.8 86.0 105  4096 x 5120    -   179  133  115 92.8 105
    // (the last two's 272 and 320 blocks of 256 x 256 are a second round of a few: the rule does not look at it)
    // Few blocks of K do not pay for a second group's sums: 64 x 64 with two groups and with one (stages of two blocks)
    // 64 x 2048 x 1024 5.0 and 4.5, 33 x 4096 x 2048 6.5 and 6.0, 64 x 8192 x 4096 10.3 and 13.7
    if (T <= 16 && N <= 8192) return launch_fp8_skinny<1>(a, s);
    if (T <= 32 && N <= 4096) return launch_fp8_skinny<2>(a, s);
    const auto tiles = [&](int64_t rows, int64_t cols) { return (T + rows - 1) / rows * ((N + cols - 1) / cols); };
    if (tiles(64, 64) <= 256) return K > 2048 ? launch_fp8<2, 2, 1, 2>(a, s) : launch_fp8<2, 2, 2, 1>(a, s);
    if (tiles(64, 128) <= 256) return launch_fp8<2, 4, 1, 2>(a, s);
    if (tiles(64, 128) <= 512) return launch_fp8<2, 4, 1, 1>(a, s);
    if (tiles(128, 128) <= 512) return launch_fp8<4, 4, 1, 1>(a, s);
    return launch_fp8_wide(a, s);
}
