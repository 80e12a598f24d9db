// mx_gemm: the dense product of MX operands around the experts,
//   out[t, n] = sum_k a[t, k] * w[n, k]
// on gfx950's block-scaled MFMA, which takes one e8m0 scale per 32 elements
// along K of either operand: the codes go to the matrix cores as they are
// stored, and the scales as bytes of a register (op_sel picks the byte).
//
// MFMA operands (32 x 32 x 64 and 16 x 16 x 128; a lane's row r and group g):
// a lane's e2m1 operand is one block, block g of the step (16 bytes); its e4m3
// operand is 16 bytes at element 16 g and 16 bytes at 16 (G + g), G groups, so
// blocks are spread over two lanes there; the scale register of group g is
// block g's in both. The K order is free as long as both operands and the
// scales agree on it.
//
// The matrix cores sum e2m1 products exactly (into fp32 accumulators). Of 8
// products with e4m3 values each is cut to 13 bits below the largest one's
// exponent before they are added (measured: 2^-13 beside 1 is kept, 2^-14 is
// not), which costs about 1.5e-5 of a result (3.3e-5 where one value in a
// hundred is an outlier): far below bf16's rounding, but not fp32's; hence no
// fp32 output for them.
#include "experts.hpp"
#include "mx.hpp"

namespace moe {

typedef int mfma_i8 __attribute__((ext_vector_type(8)));
typedef float mx_f16v __attribute__((ext_vector_type(16)));

struct MgArgs {
    const uint8_t* a;
    const uint8_t* a_sf;
    const uint8_t* w;
    const uint8_t* w_sf;
    int T, N, K;
    void* out;
    int64_t out_stride;     // elements
    int out_f32;
    int out_vec;            // rows of out start at multiples of 16 bytes
};

// A lane's operand of one MFMA.
template <int FMT>
struct MxFrag {
    uint4 q[FMT == MOE_MX_E2M1 ? 1 : 2];
    __device__ __forceinline__ mfma_i8 reg() const {
        if constexpr (FMT == MOE_MX_E2M1) return mfma_i8{(int)q[0].x, (int)q[0].y, (int)q[0].z, (int)q[0].w, 0, 0, 0, 0};
        else return mfma_i8{(int)q[0].x, (int)q[0].y, (int)q[0].z, (int)q[0].w,
                            (int)q[1].x, (int)q[1].y, (int)q[1].z, (int)q[1].w};
    }
};

template <int FMT>
constexpr int mfma_fmt() { return FMT == MOE_MX_E2M1 ? 4 : 0; }

// The scale bytes of blocks [b0, b0 + 4) of a row with nb blocks, 0 behind the
// last. ALIGNED: nb % 4 == 0, so the four lie in one aligned word.
template <bool ALIGNED>
__device__ __forceinline__ uint32_t scale_word(const uint8_t* row, int b0, int nb) {
    if constexpr (ALIGNED) {
        return b0 < nb ? *reinterpret_cast<const uint32_t*>(row + b0) : 0u;
    } else {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (b0 + i < nb) w |= (uint32_t)row[b0 + i] << (8 * i);
        return w;
    }
}

__device__ __forceinline__ void store_out(const MgArgs& a, int64_t t, int n, float v) {
    if (a.out_f32) reinterpret_cast<float*>(a.out)[t * a.out_stride + n] = v;
    else reinterpret_cast<uint16_t*>(a.out)[t * a.out_stride + n] = (uint16_t)f32_to_bf16(v);
}

// ------------------------------------------------------------------ few tokens
// Up to 64 tokens the product is a stream of the weights. A workgroup owns 16
// columns and its 8 waves split K, so that N = 4096 columns already put a
// workgroup on each CU and all of a column's weights are in flight at once;
// the waves' sums are added through LDS in wave order. 16 x 16 x 128 MFMAs
// with the weights as rows: a lane ends up with 4 consecutive columns of one
// token. The tokens' codes are read by every workgroup, from the L2.
constexpr int kSkWaves = 8;

template <int FMT>
__device__ __forceinline__ MxFrag<FMT> load_frag16(const uint8_t* row, int step, int g, int nb, int K) {
    MxFrag<FMT> f;
    if constexpr (FMT == MOE_MX_E2M1) {
        const int b = 4 * step + g;
        f.q[0] = b < nb ? *reinterpret_cast<const uint4*>(row + (int64_t)b * 16) : make_uint4(0u, 0u, 0u, 0u);
    } else {
        const int k0 = 128 * step + 16 * g, k1 = k0 + 64;
        f.q[0] = k0 < K ? *reinterpret_cast<const uint4*>(row + k0) : make_uint4(0u, 0u, 0u, 0u);
        f.q[1] = k1 < K ? *reinterpret_cast<const uint4*>(row + k1) : make_uint4(0u, 0u, 0u, 0u);
    }
    return f;
}

template <int FA, int FW, int TM, bool ALIGNED>
__global__ void __launch_bounds__(64 * kSkWaves) mx_gemm_skinny_kernel(MgArgs a) {
    constexpr int U = TM == 4 ? 2 : 4;      // steps whose loads issue together
    __shared__ floatx4 s_sum[kSkWaves][TM][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16, nb = a.K >> 5;
    const int nrow = n0 + r < a.N ? n0 + r : a.N - 1;
    const uint8_t* wrow = a.w + nrow * mx_bytes(a.K, FW);
    const uint8_t* wsf = a.w_sf + (int64_t)nrow * nb;
    const uint8_t *arow[TM], *asf[TM];
#pragma unroll
    for (int m = 0; m < TM; ++m) {
        const int t = 16 * m + r < a.T ? 16 * m + r : a.T - 1;
        arow[m] = a.a + t * mx_bytes(a.K, FA);
        asf[m] = a.a_sf + (int64_t)t * nb;
    }
    floatx4 acc[TM];
#pragma unroll
    for (int m = 0; m < TM; ++m) acc[m] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    const int steps = (a.K + 127) / 128, per = (steps + kSkWaves - 1) / kSkWaves;
    const int s0 = wave * per, s1 = s0 + per < steps ? s0 + per : steps;
    for (int s = s0; s < s1; s += U) {
        MxFrag<FW> fw[U];
        MxFrag<FA> fa[U][TM];
        uint32_t sw[U], sa[U][TM];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // steps behind s1 belong to the next wave: zeros here
            const int lim = s + u < s1 ? nb : 0, limk = s + u < s1 ? a.K : 0;
            fw[u] = load_frag16<FW>(wrow, s + u, g, lim, limk);
            sw[u] = scale_word<ALIGNED>(wsf, 4 * (s + u), lim);
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                fa[u][m] = load_frag16<FA>(arow[m], s + u, g, lim, limk);
                sa[u][m] = scale_word<ALIGNED>(asf[m], 4 * (s + u), lim);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int m = 0; m < TM; ++m)
                acc[m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    fw[u].reg(), fa[u][m].reg(), acc[m], mfma_fmt<FW>(), mfma_fmt<FA>(), 0,
                    (int)(sw[u] >> (8 * g)), 0, (int)(sa[u][m] >> (8 * g)));
    }
#pragma unroll
    for (int m = 0; m < TM; ++m) s_sum[wave][m][lane] = acc[m];
    __syncthreads();
    if (wave >= TM) return;
    floatx4 sum = s_sum[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kSkWaves; ++w) sum += s_sum[w][wave][lane];
    const int t = 16 * wave + r, n = n0 + 4 * g;
    if (t >= a.T) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < a.N) store_out(a, t, n + i, sum[i]);
}

// ------------------------------------------------------------------ many tokens
// A workgroup of 4 waves (2 x 2) computes a 64 MW x 64 NW block of the output,
// a wave MW x NW MFMA tiles of 32 x 32, over K in stages of 128 bytes a token
// row (256 elements in e2m1, 128 in e4m3). Both operands go from global memory
// to LDS directly (16 bytes a lane, two stage buffers): the copy of stage
// s + 2 is issued when every wave has read the last of stage s, behind the
// stage's one barrier, and that barrier stands before the stage's last step's
// MFMAs, whose operands are in registers by then, so the matrix cores run
// through it. A step's operands are read from LDS during the step before.
//
// LDS rows are 128 bytes (64 for e2m1 weights beside e4m3 tokens) without
// padding, which the direct copies do not allow; the 16-byte chunks of a row
// are XOR-permuted so that 16 consecutive rows' reads of one chunk spread over
// all 64 banks.
template <int FA, int FW>
struct MgShape {
    static constexpr int kElems = FA == MOE_MX_E2M1 ? 256 : 128;     // K elements a stage
    static constexpr int kSteps = kElems / 64;
    static constexpr int kABytes = 128;
    static constexpr int kWBytes = FW == MOE_MX_E2M1 ? kElems / 2 : kElems;
};

template <int BYTES>
__device__ __forceinline__ int mg_swizzle(int chunk, int row) {
    if constexpr (BYTES == 128) return chunk ^ (row & 7) ^ ((row >> 3) & 1);
    else return chunk ^ ((row >> 2) & 3);
}

// One operand's share of a stage copy by one wave: instruction q of the wave
// covers 1 KB, the rows [ROWS_PER (4 q + wave), + ROWS_PER).
template <int BYTES, int COPIES>
struct MgCopy {
    static constexpr int kChunks = BYTES / 16, kRowsPer = 64 / kChunks;
    u32x4 rsrc;
    uint32_t off[COPIES];
    int chunk;              // of the row, this lane's
    __device__ __forceinline__ void init(const uint8_t* base, int64_t row_bytes, int rows_left, int wave, int lane) {
        rsrc = buffer_desc(base);
        // kRowsPer (4 q + wave) keeps the swizzle of the rows the same for all q
        const int r0 = kRowsPer * wave + lane / kChunks;
        chunk = mg_swizzle<BYTES>(lane % kChunks, r0);
#pragma unroll
        for (int q = 0; q < COPIES; ++q) {
            const int r = r0 + 4 * kRowsPer * q;
            off[q] = (uint32_t)((r < rows_left ? r : rows_left - 1) * row_bytes + chunk * 16);
        }
    }
    // stage s into LDS at lds; row_bytes: chunks from there on (the last stage's
    // tail) are out of the descriptor's range and arrive as zeros
    __device__ __forceinline__ void issue(uint32_t lds, int s, int wave, int row_bytes) const {
        const bool in = s * BYTES + chunk * 16 < row_bytes;
#pragma unroll
        for (int q = 0; q < COPIES; ++q)
            lds_copy16(rsrc, __builtin_amdgcn_readfirstlane(lds + (4 * q + wave) * 1024),
                       in ? off[q] : 0x80000000u, (uint32_t)(s * BYTES));
    }
};

template <int FMT, int BYTES, int BLOCK_STRIDE>
__device__ __forceinline__ MxFrag<FMT> mg_read(const uint8_t* rows, int row, int g, int step) {
    MxFrag<FMT> f;
    const uint8_t* p = rows + row * BYTES;
    if constexpr (FMT == MOE_MX_E2M1) {
        // block of (group, step): 4 g + step where a stage has 4 steps (its four
        // scales are one word), else 2 step + g, e4m3's order
        const int c = BLOCK_STRIDE == 4 ? 4 * g + step : 2 * step + g;
        f.q[0] = *reinterpret_cast<const uint4*>(p + 16 * mg_swizzle<BYTES>(c, row));
    } else {
        f.q[0] = *reinterpret_cast<const uint4*>(p + 16 * mg_swizzle<BYTES>(4 * step + g, row));
        f.q[1] = *reinterpret_cast<const uint4*>(p + 16 * mg_swizzle<BYTES>(4 * step + 2 + g, row));
    }
    return f;
}

template <int FA, int FW, int MW, int NW, int STEP>
__device__ __forceinline__ void mg_mfma(mx_f16v (&acc)[MW][NW], const MxFrag<FA> (&fa)[MW], const MxFrag<FW> (&fw)[NW],
                                        const uint32_t (&sa)[MW], const uint32_t (&sw)[NW]) {
    constexpr int sel = MgShape<FA, FW>::kSteps == 4 ? STEP : 2 * STEP;
#pragma unroll
    for (int m = 0; m < MW; ++m)
#pragma unroll
        for (int n = 0; n < NW; ++n)
            acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[n].reg(), fa[m].reg(), acc[m][n],
                                                                       mfma_fmt<FW>(), mfma_fmt<FA>(), sel, (int)sw[n],
                                                                       sel, (int)sa[m]);
}

template <int FA, int FW, int MW, int NW, bool ALIGNED>
__global__ void __launch_bounds__(256, MW * NW >= 16 ? 1 : 2) mx_gemm_tiled_kernel(MgArgs a) {
    using S = MgShape<FA, FW>;
    constexpr int BM = 64 * MW, BN = 64 * NW, kStageBytes = BM * S::kABytes + BN * S::kWBytes;
    constexpr int kOutRow = 32 * NW * 4 + 16;           // one token's columns of a wave in the epilogue, fp32
    constexpr int kLds = 2 * kStageBytes > 4 * 32 * kOutRow ? 2 * kStageBytes : 4 * 32 * kOutRow;
    __shared__ __align__(16) uint8_t lds[kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, g = lane >> 5, wm = wave >> 1, wn = wave & 1;

    // Blocks of the output to workgroups: each XCD (workgroups are dealt to the 8
    // round robin) gets a contiguous run of them, and a run goes through groups
    // of 8 rows of blocks column by column, so that an XCD's L2 holds what its
    // workgroups share.
    const int mt = (a.T + BM - 1) / BM, nt = (a.N + BN - 1) / BN, tiles = mt * nt;
    const int x = blockIdx.x & 7, per = tiles >> 3, more = tiles & 7;
    const int id = x * per + (x < more ? x : more) + (int)(blockIdx.x >> 3);
    const int group = id / (8 * nt), gm0 = group * 8, gh = mt - gm0 < 8 ? mt - gm0 : 8, in = id - gm0 * nt;
    const int64_t m0 = (int64_t)(gm0 + in % gh) * BM, n0 = (int64_t)(in / gh) * BN;

    const int nb = a.K >> 5, a_row = (int)mx_bytes(a.K, FA), w_row = (int)mx_bytes(a.K, FW);
    const int stages = (a.K + S::kElems - 1) / S::kElems;
    MgCopy<S::kABytes, BM * S::kABytes / 4096> ca;
    MgCopy<S::kWBytes, BN * S::kWBytes / 4096> cw;
    ca.init(a.a + m0 * a_row, a_row, (int)(a.T - m0 < BM ? a.T - m0 : BM), wave, lane);
    cw.init(a.w + n0 * w_row, w_row, (int)(a.N - n0 < BN ? a.N - n0 : BN), wave, lane);
    const uint32_t lds0 = lds_addr(lds);
    auto copy = [&](int s) {
        const uint32_t at = lds0 + (s & 1) * kStageBytes;
        ca.issue(at, s, wave, a_row);
        cw.issue(at + BM * S::kABytes, s, wave, w_row);
    };
    const uint8_t *pa_sf[MW], *pw_sf[NW];
#pragma unroll
    for (int m = 0; m < MW; ++m) {
        const int64_t t = m0 + 32 * (wm * MW + m) + r;
        pa_sf[m] = a.a_sf + (t < a.T ? t : a.T - 1) * nb;
    }
#pragma unroll
    for (int n = 0; n < NW; ++n) {
        const int64_t c = n0 + 32 * (wn * NW + n) + r;
        pw_sf[n] = a.w_sf + (c < a.N ? c : a.N - 1) * nb;
    }
    // a stage's scales of the lane's rows: the word of group g's 4 blocks, or
    // (2 steps) the stage's word moved so that step s's byte is 2 s
    auto scales = [&](int s, uint32_t (&sa)[MW], uint32_t (&sw)[NW]) {
        const int b0 = s * (S::kElems / 32) + (S::kSteps == 4 ? 4 * g : 0), shift = S::kSteps == 4 ? 0 : 8 * g;
#pragma unroll
        for (int m = 0; m < MW; ++m) sa[m] = scale_word<ALIGNED>(pa_sf[m], b0, nb) >> shift;
#pragma unroll
        for (int n = 0; n < NW; ++n) sw[n] = scale_word<ALIGNED>(pw_sf[n], b0, nb) >> shift;
    };
    MxFrag<FA> fa[2][MW];
    MxFrag<FW> fw[2][NW];
    auto read = [&](int s, int step, int f) {
        const uint8_t* pa = lds + (s & 1) * kStageBytes;
        const uint8_t* pw = pa + BM * S::kABytes;
#pragma unroll
        for (int m = 0; m < MW; ++m)
            fa[f][m] = mg_read<FA, S::kABytes, S::kSteps>(pa, 32 * (wm * MW + m) + r, g, step);
#pragma unroll
        for (int n = 0; n < NW; ++n)
            fw[f][n] = mg_read<FW, S::kWBytes, S::kSteps>(pw, 32 * (wn * NW + n) + r, g, step);
    };

    mx_f16v acc[MW][NW];
#pragma unroll
    for (int m = 0; m < MW; ++m)
#pragma unroll
        for (int n = 0; n < NW; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.0f;

    uint32_t sa[2][MW], sw[2][NW];
    copy(0);
    scales(0, sa[0], sw[0]);
    if (stages > 1) copy(1);
    __builtin_amdgcn_s_waitcnt(vmcnt_at_most(0));
    __syncthreads();
    read(0, 0, 0);
    for (int s = 0; s < stages; ++s) {
        if (s + 1 < stages) scales(s + 1, sa[1], sw[1]);
        if constexpr (S::kSteps == 4) {
            read(s, 1, 1);
            mg_mfma<FA, FW, MW, NW, 0>(acc, fa[0], fw[0], sa[0], sw[0]);
            read(s, 2, 0);
            mg_mfma<FA, FW, MW, NW, 1>(acc, fa[1], fw[1], sa[0], sw[0]);
            read(s, 3, 1);
            mg_mfma<FA, FW, MW, NW, 2>(acc, fa[0], fw[0], sa[0], sw[0]);
        } else {
            read(s, 1, 1);
            mg_mfma<FA, FW, MW, NW, 0>(acc, fa[0], fw[0], sa[0], sw[0]);
        }
        // every wave's operands of the stage's last step are in registers, and
        // the next stage's copies have landed
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (s + 2 < stages) copy(s + 2);
        if (s + 1 < stages) read(s + 1, 0, 0);
        mg_mfma<FA, FW, MW, NW, S::kSteps - 1>(acc, fa[1], fw[1], sa[0], sw[0]);
#pragma unroll
        for (int m = 0; m < MW; ++m) sa[0][m] = sa[1][m];
#pragma unroll
        for (int n = 0; n < NW; ++n) sw[0][n] = sw[1][n];
    }

    // Epilogue: a lane holds 4 consecutive columns of one token at a time. Each
    // wave turns 32 tokens of its columns through its own part of the LDS (free
    // since the last barrier) and stores whole 16-byte pieces of a token's row.
    uint8_t* slab = lds + wave * 32 * kOutRow;
    const int es = a.out_f32 ? 4 : 2, piece = 16 / es, pieces = 32 * NW / piece;
#pragma unroll
    for (int m = 0; m < MW; ++m) {
        wave_lds_sync();
#pragma unroll
        for (int n = 0; n < NW; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = 32 * n + 8 * q + 4 * g;
                const mx_f16v& v = acc[m][n];
                if (a.out_f32)
                    *reinterpret_cast<floatx4*>(slab + r * kOutRow + c * 4) =
                        floatx4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                else
                    *reinterpret_cast<uint2*>(slab + r * kOutRow + c * 2) =
                        make_uint2(f32_to_bf16(v[4 * q]) | (f32_to_bf16(v[4 * q + 1]) << 16),
                                   f32_to_bf16(v[4 * q + 2]) | (f32_to_bf16(v[4 * q + 3]) << 16));
            }
        wave_lds_sync();
        for (int i = lane; i < 32 * pieces; i += 64) {
            const int tr = i / pieces, c = (i - tr * pieces) * piece;
            const int64_t t = m0 + 32 * (wm * MW + m) + tr, n = n0 + 32 * NW * wn + c;
            if (t >= a.T || n >= a.N) continue;
            const uint8_t* src = slab + tr * kOutRow + c * es;
            uint8_t* dst = (uint8_t*)a.out + (t * a.out_stride + n) * es;
            if (a.out_vec && n + piece <= a.N) {
                *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
            } else {
                for (int j = 0; j < piece && n + j < a.N; ++j) {
                    if (a.out_f32) reinterpret_cast<float*>(dst)[j] = reinterpret_cast<const float*>(src)[j];
                    else reinterpret_cast<uint16_t*>(dst)[j] = reinterpret_cast<const uint16_t*>(src)[j];
                }
            }
        }
    }
}

template <int FA, int FW, bool ALIGNED>
int launch_mx_gemm(const MgArgs& a, hipStream_t s) {
    const char* name = "mx_gemm";
    if (a.T <= 64) {
        const dim3 g((unsigned)((a.N + 15) / 16)), b(64 * kSkWaves);
        if (a.T <= 16) hipLaunchKernelGGL((mx_gemm_skinny_kernel<FA, FW, 1, ALIGNED>), g, b, 0, s, a);
        else if (a.T <= 32) hipLaunchKernelGGL((mx_gemm_skinny_kernel<FA, FW, 2, ALIGNED>), g, b, 0, s, a);
        else hipLaunchKernelGGL((mx_gemm_skinny_kernel<FA, FW, 4, ALIGNED>), g, b, 0, s, a);
        return check_launch(name);
    }
    const auto tiles = [&](int bm, int bn) { return (int64_t)((a.T + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
    if (tiles(64, 64) > 0x7FFFFFFF) return fail(MOE_EUNSUPPORTED, "%s: too many output tiles", name);
    // the largest tile that still gives every CU one
    if (tiles(256, 256) >= 192)
        hipLaunchKernelGGL((mx_gemm_tiled_kernel<FA, FW, 4, 4, ALIGNED>), dim3((unsigned)tiles(256, 256)), dim3(256), 0, s, a);
    else if (tiles(128, 128) >= 192)
        hipLaunchKernelGGL((mx_gemm_tiled_kernel<FA, FW, 2, 2, ALIGNED>), dim3((unsigned)tiles(128, 128)), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((mx_gemm_tiled_kernel<FA, FW, 1, 1, ALIGNED>), dim3((unsigned)tiles(64, 64)), dim3(256), 0, s, a);
    return check_launch(name);
}

template <int FA, int FW>
int launch_mx_gemm(const MgArgs& a, hipStream_t s) {
    return (a.K / 32) % 4 == 0 ? launch_mx_gemm<FA, FW, true>(a, s) : launch_mx_gemm<FA, FW, false>(a, s);
}

}  // namespace moe

extern "C" int mx_gemm(const uint8_t* a_codes, const uint8_t* a_sf, int a_fmt, const uint8_t* w_codes,
                       const uint8_t* w_sf, int w_fmt, int T, int N, int K, void* out, int64_t out_row_stride,
                       int out_dtype, void* stream) {
    using namespace moe;
    const char* name = "mx_gemm";
    if (T < 0 || N < 0 || K < 0) return fail(MOE_EINVAL, "%s: negative size T=%d N=%d K=%d", name, T, N, K);
    if (!mx_fmt_ok(a_fmt) || !mx_fmt_ok(w_fmt))
        return fail(MOE_EINVAL, "%s: formats %d, %d are not MOE_MX_E2M1 or MOE_MX_E4M3", name, a_fmt, w_fmt);
    if (out_dtype != MOE_BF16 && out_dtype != MOE_F32)
        return fail(MOE_EINVAL, "%s: dtype %d is neither MOE_BF16 nor MOE_F32", name, out_dtype);
    if (a_fmt == MOE_MX_E2M1 && w_fmt == MOE_MX_E4M3)
        return fail(MOE_EUNSUPPORTED, "%s: e2m1 activations with e4m3 weights", name);
    if (out_dtype == MOE_F32 && a_fmt == MOE_MX_E4M3)
        return fail(MOE_EUNSUPPORTED, "%s: fp32 output needs e2m1 operands", name);
    if (K < kMxBlock || K % kMxBlock || K > MOE_MAX_MX_K)
        return fail(MOE_EUNSUPPORTED, "%s: K=%d must be a multiple of 32 in [32, %d]", name, K, MOE_MAX_MX_K);
    if (T == 0 || N == 0) return MOE_OK;
    if (!a_codes || !a_sf || !w_codes || !w_sf || !out) return fail(MOE_EINVAL, "%s: NULL pointer", name);
    if (!aligned16(a_codes) || !aligned16(a_sf) || !aligned16(w_codes) || !aligned16(w_sf) || !aligned16(out))
        return fail(MOE_EINVAL, "%s: pointers must be 16-byte aligned", name);
    if (out_row_stride < N) return fail(MOE_EINVAL, "%s: out row stride %lld must be >= N", name, (long long)out_row_stride);
    MgArgs a{a_codes, a_sf, w_codes, w_sf, T, N, K, out, out_row_stride, out_dtype == MOE_F32 ? 1 : 0,
             (out_row_stride * (out_dtype == MOE_F32 ? 4 : 2)) % 16 == 0 ? 1 : 0};
    hipStream_t s = (hipStream_t)stream;
    if (a_fmt == MOE_MX_E2M1) return launch_mx_gemm<MOE_MX_E2M1, MOE_MX_E2M1>(a, s);
    if (w_fmt == MOE_MX_E2M1) return launch_mx_gemm<MOE_MX_E4M3, MOE_MX_E2M1>(a, s);
    return launch_mx_gemm<MOE_MX_E4M3, MOE_MX_E4M3>(a, s);
}
