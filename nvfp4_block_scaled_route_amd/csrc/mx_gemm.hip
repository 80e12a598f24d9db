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
// The matrix cores add e2m1 products whole (into fp32 accumulators, which round
// once a step). Of 8 products with e4m3 values each is cut to 13 bits below the largest one's
// exponent before they are added (measured: 2^-13 beside 1 is kept, 2^-14 is
// not), which costs about 1.5e-5 of a result (3.3e-5 where one value in a
// hundred is an outlier): far below bf16's rounding, but not fp32's; hence no
// fp32 output for them.
//
// The compiler may sink MFMAs into a divergent branch that alone uses their
// result, where lanes are off and their operands lost: both kernels use every
// accumulator in all lanes (a write to the LDS), and branch behind that.
#include <type_traits>

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
// Up to 32 tokens the product is a stream of the weights. A workgroup owns 16
// columns (TN = 1) and its 8 waves split K, so that N = 4096 columns already put
// a workgroup on each CU and all of a column's weights are in flight at once (4
// or 16 waves: the same or slower); the waves' sums are added through LDS in
// wave order. With more columns it owns 32 (TN = 2), which reads the tokens half
// as often (64: slower, 8 x 8192 x 4096 9.2 us against 7.1). 16 x 16 x 128 MFMAs
// with the weights as rows: a lane ends up with 4 consecutive columns of one
// token. The tokens' codes are read by every workgroup, from the L2.
//
// The number of load instructions bounds it: with a load a step for the scales
// 8 x 4096 x 4096 e4m3 x e2m1 took 5.9 us, with one for four steps 4.9 (1.9
// TB/s); 8 x 16384 x 4096 16.8 and 12.9, and 10.6 (3.4 TB/s) with 32 columns.
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

template <int FA, int FW, int TM, int TN, bool ALIGNED>
__global__ void __launch_bounds__(64 * kSkWaves) mx_gemm_skinny_kernel(MgArgs a) {
    constexpr int U = 4;                    // steps whose loads issue together
    __shared__ floatx4 s_sum[kSkWaves][TM * TN][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * (16 * TN), nb = a.K >> 5;
    const uint8_t *wrow[TN], *wsf[TN], *arow[TM], *asf[TM];
#pragma unroll
    for (int n = 0; n < TN; ++n) {
        const int row = n0 + 16 * n + r < a.N ? n0 + 16 * n + r : a.N - 1;
        wrow[n] = a.w + row * mx_bytes(a.K, FW);
        wsf[n] = a.w_sf + (int64_t)row * nb;
    }
#pragma unroll
    for (int m = 0; m < TM; ++m) {
        const int t = 16 * m + r < a.T ? 16 * m + r : a.T - 1;
        arow[m] = a.a + t * mx_bytes(a.K, FA);
        asf[m] = a.a_sf + (int64_t)t * nb;
    }
    floatx4 acc[TM][TN];
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int n = 0; n < TN; ++n) acc[m][n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    const int steps = (a.K + 127) / 128, per = (steps + kSkWaves - 1) / kSkWaves;
    const int s0 = wave * per, s1 = s0 + per < steps ? s0 + per : steps;
    for (int s = s0; s < s1; s += U) {
        MxFrag<FW> fw[U][TN];
        MxFrag<FA> fa[U][TM];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // steps behind s1 belong to the next wave: zeros here
            const int lim = s + u < s1 ? nb : 0, limk = s + u < s1 ? a.K : 0;
#pragma unroll
            for (int n = 0; n < TN; ++n) fw[u][n] = load_frag16<FW>(wrow[n], s + u, g, lim, limk);
#pragma unroll
            for (int m = 0; m < TM; ++m) fa[u][m] = load_frag16<FA>(arow[m], s + u, g, lim, limk);
        }
        // The scales of U steps in one load a row: lane group g takes step s + g's
        // four and hands them round.
        static_assert(U == 4, "a step a lane group");
        const int lim = s + g < s1 ? nb : 0;
        uint32_t xw[TN], xa[TM];
#pragma unroll
        for (int n = 0; n < TN; ++n) xw[n] = scale_word<ALIGNED>(wsf[n], 4 * (s + g), lim);
#pragma unroll
        for (int m = 0; m < TM; ++m) xa[m] = scale_word<ALIGNED>(asf[m], 4 * (s + g), lim);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int sw[TN], sa[TM];
#pragma unroll
            for (int n = 0; n < TN; ++n) sw[n] = (int)((uint32_t)__builtin_amdgcn_ds_bpermute(4 * (16 * u + r), (int)xw[n]) >> (8 * g));
#pragma unroll
            for (int m = 0; m < TM; ++m) sa[m] = (int)((uint32_t)__builtin_amdgcn_ds_bpermute(4 * (16 * u + r), (int)xa[m]) >> (8 * g));
#pragma unroll
            for (int m = 0; m < TM; ++m)
#pragma unroll
                for (int n = 0; n < TN; ++n)
                    acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        fw[u][n].reg(), fa[u][m].reg(), acc[m][n], mfma_fmt<FW>(), mfma_fmt<FA>(), 0, sw[n], 0, sa[m]);
        }
    }
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int n = 0; n < TN; ++n) s_sum[wave][m * TN + n][lane] = acc[m][n];
    __syncthreads();
    if (wave >= TM * TN) return;
    floatx4 sum = s_sum[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kSkWaves; ++w) sum += s_sum[w][wave][lane];
    const int t = 16 * (wave / TN) + r, n = n0 + 16 * (wave % TN) + 4 * g;
    if (t >= a.T) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < a.N) store_out(a, t, n + i, sum[i]);
}

// ------------------------------------------------------------------ many tokens
// A workgroup of 4 waves (2 x 2) computes a 64 MW x 64 NW block of the output,
// a wave MW x NW MFMA tiles of 32 x 32, over K in stages of 256 elements or 128
// (4 or 2 MFMA steps), as far as it fits whole cache lines of the rows: with
// 64-byte pieces of e2m1 rows a stage, each line was fetched from the L2 twice
// (4096 x 4096 x 4096: 51.7 us, with whole lines 45.2).
//
// Codes and scales go from global memory to LDS directly, into a ring of kRing
// stage buffers. A stage has one barrier, before its last step's MFMAs: every
// wave's reads of the stage are in registers by then (a step's operands are
// read during the step before) and the next stage's copies have landed; after
// it, the copies of stage s + kRing go into the buffer just freed, spread over
// the MFMAs that follow. So the matrix cores run through the barrier, and the
// wait before it leaves the younger stages' copies in flight (vmcnt counts them
// in order, and every wave issues the same number).
//
// LDS rows are 64, 128 or 256 bytes without padding, which the direct copies do
// not allow; the 16-byte chunks of a row are XOR-permuted so that 16 consecutive
// rows' reads of one chunk spread over all 64 banks.
//
// 4096 x 4096 x 4096, from one GPU to another: e2m1 39 to 43 us (3.2 to 3.5
// PFLOP/s; the MFMAs alone 21.8 on random data, where the chip's power holds the
// matrix unit at 6.3 PFLOP/s, and 8.5 on zeros), fp32 output 47, e4m3 x e2m1 59
// to 65 us (2.2 PFLOP/s), e4m3 x e4m3 66.

// A row's scales travel in chunks: 32 of them (1024 elements) as two 16-byte
// pieces where their words are aligned (K / 32 a multiple of 4, at least 16),
// else 24 (768 elements) as the 8 aligned words from the one that holds the
// chunk's first byte; the last such word of the array may reach 3 bytes past it.
// Every stage's own few bytes would touch as many cache lines as the codes do.
// PIECES: of an aligned chunk.
template <int PIECES, bool ALIGNED>
struct MgScale {
    static constexpr int kBytes = ALIGNED ? 16 * PIECES : 24, kRow = ALIGNED ? 16 * PIECES : 32;      // of a row, in memory and in LDS
};

template <int FA, int FW, int MW, int NW, bool ALIGNED>
struct MgShape {
    static constexpr int kBM = 64 * MW, kBN = 64 * NW;
    // K of a stage: 256 with e2m1 tokens (128 bytes of a row), and with e4m3 tokens
    // in the blocks below 128 x 128; in the wider ones LDS would hold too few such
    // stages (e4m3 x e2m1 2048 x 4096 x 4096 in 128-wide blocks: 48.3 us with 256,
    // 41.2 with 128). e4m3 x e4m3 was not timed with 128 in the small blocks: its 64
    // x 128 block with 256 takes nearly all of a CU's LDS.
    static constexpr int kElems = FA == MOE_MX_E2M1 || MW * NW < 4 ? 256 : 128;
    static constexpr int kSteps = kElems / 64;
    static constexpr int kABytes = FA == MOE_MX_E2M1 ? kElems / 2 : kElems;
    static constexpr int kWBytes = FW == MOE_MX_E2M1 ? kElems / 2 : kElems;
    static constexpr int kACopies = kBM * kABytes / 4096, kWCopies = kBN * kWBytes / 4096;   // a wave's, per stage
    static constexpr int kAll = kACopies + kWCopies;
    static constexpr int kW = kBM * kABytes, kStage = kW + kBN * kWBytes;
    static constexpr int kPieces = MW * NW < 16 ? 2 : 1;
    using Sf = MgScale<kPieces, ALIGNED>;
    static constexpr int kChunk = (kBM + kBN) * Sf::kRow;     // scales, two buffers of kSpc stages each
    static constexpr int kSpc = Sf::kBytes * 32 / kElems;
    // as many stages, 2 to 6, as leave a CU 2 workgroups (1 of the widest): what
    // is in flight hides the memory's latency where the blocks are small. A chunk
    // of scales overwrites the last but one, whose stages must be past (ring of
    // at most kSpc + 1).
    static constexpr int kPerCu = MW * NW >= 16 || 2 * (2 * kStage + 2 * kChunk) > 160 * 1024 ? 1 : 2;
    static constexpr int kFit = (160 * 1024 / kPerCu - 2 * kChunk) / kStage, kMax = kSpc + 1 < 6 ? kSpc + 1 : 6;
    static constexpr int kRing = kFit < kMax ? kFit : kMax;
    static constexpr int kSf = kRing * kStage, kLds = kSf + 2 * kChunk;
    static_assert(kRing >= 2 && (kRing - 1) * kAll < 64, "ring of stages");
};

template <int BYTES>
__device__ __forceinline__ int mg_swizzle(int chunk, int row) {
    if constexpr (BYTES == 256) return chunk ^ (row & 15);
    else if constexpr (BYTES == 128) return chunk ^ (row & 7) ^ ((row >> 3) & 1);
    else return chunk ^ ((row >> 2) & 3);
}

// Direct-to-LDS load of one word a lane, as lds_copy16.
__device__ __forceinline__ void lds_copy4(u32x4 rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
    asm volatile("buffer_load_dword %0, %1, %2 offen lds" :: "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds) : "memory");
}

// One operand's codes: instruction q of a wave copies 1 KB, the rows
// [kRowsPer (4 q + wave), + kRowsPer) of a stage.
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
    // instruction q of stage s into LDS at lds. Chunks from row_bytes on (the
    // last stage's tail, stages behind it) are out of the descriptor's range and
    // arrive as zeros.
    __device__ __forceinline__ void issue(uint32_t lds, int s, int q, int wave, int row_bytes) const {
        lds_copy16(rsrc, __builtin_amdgcn_readfirstlane(lds + (4 * q + wave) * 1024),
                   s * BYTES + chunk * 16 < row_bytes ? off[q] : 0x80000000u, (uint32_t)(s * BYTES));
    }
};

// One operand's scales, aligned. Blocks of few rows take less than one
// instruction a wave: waves then repeat each other's.
template <int ROWS, int PIECES, bool ALIGNED>
struct MgScaleCopy {
    static constexpr int kRowsPer = 64 / PIECES, kParts = ROWS / kRowsPer, kCopies = kParts > 4 ? kParts / 4 : 1;
    u32x4 rsrc;
    uint32_t off[kCopies];  // of a lane's rows
    __device__ __forceinline__ void init(const uint8_t* base, int nb, int rows_left, int wave, int lane) {
        rsrc = buffer_desc(base);
#pragma unroll
        for (int q = 0; q < kCopies; ++q) {
            const int r = kRowsPer * ((4 * q + wave) % kParts) + lane / PIECES;
            off[q] = (uint32_t)((r < rows_left ? r : rows_left - 1) * nb);
        }
    }
    // Chunk c into LDS at lds. The piece that would pass the row's end lies
    // against it instead (MgScales goes by that).
    __device__ __forceinline__ void issue(uint32_t lds, int c, int wave, int lane, int nb) const {
        const int b = 16 * (PIECES * c + lane % PIECES), at = b < nb - 16 ? b : nb - 16;
#pragma unroll
        for (int q = 0; q < kCopies; ++q)
            lds_copy16(rsrc, __builtin_amdgcn_readfirstlane(lds + (4 * q + wave) % kParts * 1024), off[q] + at, 0u);
    }
};

// Not aligned: 8 lanes a row, each a word. Words behind a row's last scale and
// rows behind the last are zeros.
template <int ROWS, int PIECES>
struct MgScaleCopy<ROWS, PIECES, false> {
    u32x4 rsrc;
    uint32_t off;           // of a lane's first row's first word
    int row, left, skew;    // that row, the rows there are, the byte of the word at which the row starts
    __device__ __forceinline__ void init(const uint8_t* base, int nb, int rows_left, int wave, int lane) {
        rsrc = buffer_desc(base);
        row = 8 * wave + lane / 8, left = rows_left;
        off = (uint32_t)(row * nb) & ~3u, skew = row * nb & 3;
    }
    __device__ __forceinline__ void issue(uint32_t lds, int c, int wave, int lane, int nb) const {
        const int b = 24 * c + 4 * (lane % 8), end = b < nb + skew ? left : 0;
#pragma unroll
        for (int q = 0; q < ROWS / 32; ++q)     // 32 rows are whole words
            lds_copy4(rsrc, __builtin_amdgcn_readfirstlane(lds + (4 * q + wave) * 256),
                      row + 32 * q < end ? off + b : 0x80000000u, (uint32_t)(32 * q * nb));
    }
};

// A lane's operand of a step. e2m1: one block, block 4 g + step of the stage (so
// that a group's scales are one word), or beside e4m3 (PAIR) block 2 step + g,
// e4m3's order; e4m3: its share of blocks 2 step and 2 step + 1.
template <int FMT, int BYTES, bool PAIR>
__device__ __forceinline__ MxFrag<FMT> mg_read(const uint8_t* rows, int row, int g, int step) {
    MxFrag<FMT> f;
    const uint8_t* p = rows + row * BYTES;
    if constexpr (FMT == MOE_MX_E2M1) {
        f.q[0] = *reinterpret_cast<const uint4*>(p + 16 * mg_swizzle<BYTES>(PAIR ? 2 * step + g : 4 * g + step, row));
    } else {
        f.q[0] = *reinterpret_cast<const uint4*>(p + 16 * mg_swizzle<BYTES>(4 * step + g, row));
        f.q[1] = *reinterpret_cast<const uint4*>(p + 16 * mg_swizzle<BYTES>(4 * step + 2 + g, row));
    }
    return f;
}

// A stage's scales of a lane's row. read() takes what LDS holds and scales() makes
// one register of it, step s's byte at s, or with 2 steps at 2 s, zeros behind
// the row's nb blocks: apart, so that no instruction waits for the LDS between
// the reads and the MFMAs that cover them. b0: the stage's first block, c0: the
// chunk's. Not aligned, a row starts at byte `skew` of its first word.
template <int STEPS, bool PAIR, int PIECES, bool ALIGNED>
struct MgScales {
    static constexpr int kWords = PAIR && STEPS == 4 ? 2 : 1;       // of 4 blocks each
    uint2 raw[kWords];                                              // aligned: x alone
    __device__ __forceinline__ static int block(int b0, int i, int g) { return b0 + 4 * (PAIR ? i : g); }
    __device__ __forceinline__ void read(const uint8_t* row, int b0, int c0, int nb, int g) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int b = block(b0, i, g);
            if constexpr (ALIGNED) {
                const int piece = b & ~15, at = piece < nb - 16 ? piece : nb - 16;
                raw[i].x = *reinterpret_cast<const uint32_t*>(row + (PIECES == 2 ? b & 16 : 0) + (b < nb ? b - at : 0));
            } else {
                const uint32_t* w = reinterpret_cast<const uint32_t*>(row + (b - c0));
                raw[i] = make_uint2(w[0], w[1]);
            }
        }
    }
    __device__ __forceinline__ uint32_t scales(int b0, int nb, int g, int skew) const {
        uint32_t v[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int left = nb - block(b0, i, g);
            if constexpr (ALIGNED) {
                v[i] = left > 0 ? raw[i].x : 0u;
            } else {        // the next row's bytes among them
                const uint32_t w = __builtin_amdgcn_alignbyte(raw[i].y, raw[i].x, skew);
                v[i] = left >= 4 ? w : left > 0 ? w & ((1u << (8 * left)) - 1u) : 0u;
            }
        }
        if constexpr (!PAIR) return v[0];                               // blocks 4 g + step
        else if constexpr (STEPS == 2) return v[0] >> (8 * g);          // blocks g, 2 + g
        else return __builtin_amdgcn_perm(v[1], v[0], g ? 0x07050301u : 0x06040200u);   // and 4 + g, 6 + g
    }
};

// Epilogue of 32 tokens: a lane holds 4 consecutive columns of one token at a
// time. The wave turns its NW tiles through its own part of the LDS (a token's
// columns, padded by 16 bytes) and stores whole 16-byte pieces of the tokens'
// rows. NT: outputs of 256-wide blocks are past what the L2 keeps for a reader,
// non-temporal stores (4096 x 4096 x 4096 e2m1: 43.4 -> 42.6 us).
template <int NW, bool F32>
constexpr int out_row_bytes() { return 32 * NW * (F32 ? 4 : 2) + 16; }

template <int NW, bool F32, bool NT>
__device__ __forceinline__ void store_rows(const MgArgs& a, uint8_t* slab, const mx_f16v (&acc)[NW], int64_t t0, int64_t n0,
                                           int lane) {
    constexpr int kRow = out_row_bytes<NW, F32>(), kEs = F32 ? 4 : 2, kPiece = 16 / kEs, kPieces = 32 * NW / kPiece;
    const int r = lane & 31, g = lane >> 5;
    wave_lds_sync();
#pragma unroll
    for (int n = 0; n < NW; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = 32 * n + 8 * q + 4 * g;
            const mx_f16v& v = acc[n];
            if constexpr (F32)
                *reinterpret_cast<floatx4*>(slab + r * kRow + c * 4) = floatx4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            else
                *reinterpret_cast<uint2*>(slab + r * kRow + c * 2) =
                    make_uint2(bf16x2_pack(v[4 * q], v[4 * q + 1]), bf16x2_pack(v[4 * q + 2], v[4 * q + 3]));
        }
    wave_lds_sync();
#pragma unroll
    for (int j = 0; j < 32 * kPieces / 64; ++j) {
        const int i = lane + 64 * j, tr = i / kPieces, c = (i % kPieces) * kPiece;
        const int64_t t = t0 + tr, n = n0 + c;
        if (t >= a.T || n >= a.N) continue;
        const uint8_t* src = slab + tr * kRow + c * kEs;
        uint8_t* dst = (uint8_t*)a.out + (t * a.out_stride + n) * kEs;
        if (a.out_vec && n + kPiece <= a.N) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(src);
            if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(dst));
            else *reinterpret_cast<u32x4*>(dst) = v;
        } else {
            for (int e = 0; e < kPiece && n + e < a.N; ++e) {
                if constexpr (F32) reinterpret_cast<float*>(dst)[e] = reinterpret_cast<const float*>(src)[e];
                else reinterpret_cast<uint16_t*>(dst)[e] = reinterpret_cast<const uint16_t*>(src)[e];
            }
        }
    }
}

template <int FA, int FW, int MW, int NW, bool ALIGNED, bool F32>
__global__ void __launch_bounds__(256, (MgShape<FA, FW, MW, NW, ALIGNED>::kPerCu)) mx_gemm_tiled_kernel(MgArgs a) {
    using S = MgShape<FA, FW, MW, NW, ALIGNED>;
    constexpr int kOutRow = out_row_bytes<NW, F32>();
    constexpr int kLds = S::kLds > 4 * 32 * kOutRow ? S::kLds : 4 * 32 * kOutRow;
    constexpr bool kPair = FA == MOE_MX_E4M3;
    using Sf = typename S::Sf;
    constexpr int kAll = S::kAll;
    __shared__ __align__(16) uint8_t lds[kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, g = lane >> 5, wm = wave >> 1, wn = wave & 1;

    // Blocks of the output to workgroups: each XCD (workgroups are dealt to the 8
    // round robin) gets a contiguous run of them, and a run goes through groups
    // of 4 rows of blocks column by column, so that an XCD's L2 holds what its
    // workgroups share (4096 x 4096 x 4096 e2m1: 44.9 us with 8 rows, 43.4 with 4).
    const int mt = (a.T + S::kBM - 1) / S::kBM, nt = (a.N + S::kBN - 1) / S::kBN, tiles = mt * nt;
    const int x = blockIdx.x & 7, per = tiles >> 3, more = tiles & 7;
    const int id = x * per + (x < more ? x : more) + (int)(blockIdx.x >> 3);
    const int gm0 = id / (4 * nt) * 4, gh = mt - gm0 < 4 ? mt - gm0 : 4, in = id - gm0 * nt;
    const int64_t m0 = (int64_t)(gm0 + in % gh) * S::kBM, n0 = (int64_t)(in / gh) * S::kBN;

    const int nb = a.K >> 5, a_row = (int)mx_bytes(a.K, FA), w_row = (int)mx_bytes(a.K, FW);
    const int stages = (a.K + S::kElems - 1) / S::kElems;
    const int rows_m = (int)(a.T - m0 < S::kBM ? a.T - m0 : S::kBM), rows_n = (int)(a.N - n0 < S::kBN ? a.N - n0 : S::kBN);
    MgCopy<S::kABytes, S::kACopies> ca;
    MgCopy<S::kWBytes, S::kWCopies> cw;
    MgScaleCopy<S::kBM, S::kPieces, ALIGNED> csa;
    MgScaleCopy<S::kBN, S::kPieces, ALIGNED> csw;
    ca.init(a.a + m0 * a_row, a_row, rows_m, wave, lane);
    cw.init(a.w + n0 * w_row, w_row, rows_n, wave, lane);
    csa.init(a.a_sf + m0 * nb, nb, rows_m, wave, lane);
    csw.init(a.w_sf + n0 * nb, nb, rows_n, wave, lane);
    const uint32_t lds0 = lds_addr(lds);
    auto copy = [&](int s, int q0, int q1) {        // instructions [q0, q1) of stage s's kAll codes
        // a chunk of scales goes before the codes of its first stage: what waits
        // for those has waited for these
        if (q0 == 0 && s % S::kSpc == 0) {
            const uint32_t at = lds0 + S::kSf + (s / S::kSpc & 1) * S::kChunk;
            csa.issue(at, s / S::kSpc, wave, lane, nb);
            csw.issue(at + S::kBM * Sf::kRow, s / S::kSpc, wave, lane, nb);
        }
        const uint32_t at = lds0 + (s % S::kRing) * S::kStage;
#pragma unroll
        for (int q = q0; q < q1; ++q) {
            if (q < S::kACopies) ca.issue(at, s, q, wave, a_row);
            else cw.issue(at + S::kW, s, q - S::kACopies, wave, w_row);
        }
    };
    using Scales = MgScales<S::kSteps, kPair, S::kPieces, ALIGNED>;
    Scales na[MW], nw[NW];      // the next stage's, as read
    uint32_t sa[MW], sw[NW];
    const int skew = r * nb & 3;        // 32 rows are whole words
    auto read_scales = [&](int s) {
        const int c0 = s / S::kSpc * Sf::kBytes;
        const uint8_t* at = lds + S::kSf + (s / S::kSpc & 1) * S::kChunk;
#pragma unroll
        for (int m = 0; m < MW; ++m) na[m].read(at + Sf::kRow * (32 * (wm * MW + m) + r), s * (S::kElems / 32), c0, nb, g);
#pragma unroll
        for (int n = 0; n < NW; ++n) nw[n].read(at + Sf::kRow * (S::kBM + 32 * (wn * NW + n) + r), s * (S::kElems / 32), c0, nb, g);
    };
    auto take_scales = [&](int s) {
#pragma unroll
        for (int m = 0; m < MW; ++m) sa[m] = na[m].scales(s * (S::kElems / 32), nb, g, skew);
#pragma unroll
        for (int n = 0; n < NW; ++n) sw[n] = nw[n].scales(s * (S::kElems / 32), nb, g, skew);
    };
    struct Operands {
        MxFrag<FA> a[MW];
        MxFrag<FW> w[NW];
    };
    auto read = [&](int s, int step, Operands& o) {
        const uint8_t* at = lds + (s % S::kRing) * S::kStage;
#pragma unroll
        for (int n = 0; n < NW; ++n) o.w[n] = mg_read<FW, S::kWBytes, kPair>(at + S::kW, 32 * (wn * NW + n) + r, g, step);
#pragma unroll
        for (int m = 0; m < MW; ++m) o.a[m] = mg_read<FA, S::kABytes, kPair>(at, 32 * (wm * MW + m) + r, g, step);
    };

    mx_f16v acc[MW][NW];
#pragma unroll
    for (int m = 0; m < MW; ++m)
#pragma unroll
        for (int n = 0; n < NW; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.0f;
    // one MFMA row of a step; the scales' byte SEL
    auto mfma = [&](const Operands& o, int m, auto sel) {
#pragma unroll
        for (int n = 0; n < NW; ++n)
            acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(o.w[n].reg(), o.a[m].reg(), acc[m][n],
                                                                        mfma_fmt<FW>(), mfma_fmt<FA>(), sel.value,
                                                                        (int)sw[n], sel.value, (int)sa[m]);
    };
    auto mfmas = [&](const Operands& o, auto sel) {
#pragma unroll
        for (int m = 0; m < MW; ++m) mfma(o, m, sel);
        __builtin_amdgcn_sched_barrier(0);
    };

#pragma unroll
    for (int s = 0; s < S::kRing; ++s) copy(s, 0, kAll);
    Operands o0, o1;
    __builtin_amdgcn_s_waitcnt(vmcnt_at_most((S::kRing - 1) * kAll));
    __syncthreads();
    read_scales(0);
    read(0, 0, o0);
    take_scales(0);
    for (int s = 0; s < stages; ++s) {
        read(s, 1, o1);
        mfmas(o0, std::integral_constant<int, 0>());
        if constexpr (S::kSteps == 4) {
            read(s, 2, o0);
            mfmas(o1, std::integral_constant<int, 1>());
            read(s, 3, o1);
            mfmas(o0, std::integral_constant<int, 2>());
        }
        __builtin_amdgcn_s_waitcnt(vmcnt_at_most((S::kRing - 2) * kAll) & lgkmcnt_zero());
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        read_scales(s + 1);
        read(s + 1, 0, o0);
#pragma unroll
        for (int m = 0; m < MW; ++m) {
            copy(s + S::kRing, m * kAll / MW, (m + 1) * kAll / MW);
            mfma(o1, m, std::integral_constant<int, S::kSteps == 4 ? 3 : 2>());
            __builtin_amdgcn_sched_barrier(0);
        }
        take_scales(s + 1);
    }
    // the copies of the stages behind the last still write (zeros) to the LDS
    __builtin_amdgcn_s_waitcnt(vmcnt_at_most(0) & lgkmcnt_zero());
    __syncthreads();

    uint8_t* slab = lds + wave * 32 * kOutRow;
#pragma unroll
    for (int m = 0; m < MW; ++m)
        store_rows<NW, F32, (MW * NW >= 16)>(a, slab, acc[m], m0 + 32 * (wm * MW + m), n0 + 32 * NW * wn, lane);
}

template <int FA, int FW, int MW, int NW, bool ALIGNED>
void launch_mx_tiled(const MgArgs& a, hipStream_t s) {
    const int64_t tiles = (int64_t)((a.T + 64 * MW - 1) / (64 * MW)) * ((a.N + 64 * NW - 1) / (64 * NW));
    const dim3 g((unsigned)tiles), b(256);
    if constexpr (FA == MOE_MX_E2M1) {
        if (a.out_f32) {
            hipLaunchKernelGGL((mx_gemm_tiled_kernel<FA, FW, MW, NW, ALIGNED, true>), g, b, 0, s, a);
            return;
        }
    }
    hipLaunchKernelGGL((mx_gemm_tiled_kernel<FA, FW, MW, NW, ALIGNED, false>), g, b, 0, s, a);
}

template <int FA, int FW, bool ALIGNED>
int launch_mx_gemm(const MgArgs& a, hipStream_t s) {
    const char* name = "mx_gemm";
    // K = N = 4096, e4m3 x e2m1: 32 tokens 7.9 us by columns, 10.6 in 64-wide
    // blocks; 64 tokens (when 32 took 9.7) 15.6 and 11.0
    if (a.T <= 32) {
        // 32 columns a workgroup where 16 would be more than one a CU (K = 4096, e4m3 x e2m1, 16 and 32
        // columns: 8 tokens, N = 4096 4.9 and 6.3, 4224 7.1 and 6.3, 8192 7.9 and 7.0; 32 tokens,
        // 4096 7.9 and 9.3, 4608 13.0 and 9.5, 16384 23.5 and 17.7)
        const bool wide = a.N > 16 * 256;
        const dim3 g((unsigned)(((int64_t)a.N + (wide ? 31 : 15)) / (wide ? 32 : 16))), b(64 * kSkWaves);
        if (!launch_fits(g.x, b.x)) return fail(MOE_EUNSUPPORTED, "%s: too many columns", name);
        if (a.T <= 16 && wide) hipLaunchKernelGGL((mx_gemm_skinny_kernel<FA, FW, 1, 2, ALIGNED>), g, b, 0, s, a);
        else if (a.T <= 16) hipLaunchKernelGGL((mx_gemm_skinny_kernel<FA, FW, 1, 1, ALIGNED>), g, b, 0, s, a);
        else if (wide) hipLaunchKernelGGL((mx_gemm_skinny_kernel<FA, FW, 2, 2, ALIGNED>), g, b, 0, s, a);
        else hipLaunchKernelGGL((mx_gemm_skinny_kernel<FA, FW, 2, 1, ALIGNED>), g, b, 0, s, a);
        return check_launch(name);
    }
    const auto tiles = [&](int64_t bm, int64_t bn) { return (a.T + bm - 1) / bm * ((a.N + bn - 1) / bn); };
    if (!launch_fits(tiles(64, 64), 256)) return fail(MOE_EUNSUPPORTED, "%s: too many output tiles", name);
    // The widest block that fills the chip: wide blocks read less per product,
    // but a CU without one idles. us with K = 4096 (64 x 64, 64 x 128, 128 x 128,
    // 256 x 256):
    //   517 x 2048 e4m3 x e2m1   16.0  16.9  28.4  53.6     1024 x 4096  30.0  23.0  29.9  53.8
    //   1536 x 4096 e4m3 x e2m1  43.8  36.1  32.9  54.1     2048 x 4096  57.2  42.9  37.3  53.8
    //   1536 x 4096 e2m1         31.9  28.6  22.7  36.6     2800 x 4096  55.4  46.5  38.5  37.6
    // 256 x 256, a workgroup a CU, where the last round of them is filled; us, 128 x 128 and 256 x 256,
    // N = K = 4096, e2m1, by the blocks of 256 x 256:
    //   176  39.0  38.8    224  42.5  38.0    256  45.3  39.9    304  56.0  70.2    352  62.6  70.8
    //   400  75.9  71.8    512  87.9  77.4;   with K = 4128  208  53.9  49.6    256  62.2  51.3
    // Both sides of these outputs were 517 or more, and e4m3 x e4m3 is not among them. The rule
    // counts blocks and not what they hold: a thin output of many columns takes wide blocks that
    // are mostly behind its last token (e4m3 x e2m1, K = 4096: 64 x 43008 54.7 us and 64 x 65536
    // 59.2, where the bytes need 20 and 30).
    // (not e4m3 x e4m3 with scales that are not aligned, whose registers do not suffice: 4096 x 4096 x
    // 4128 160.6 us against 102.9)
    constexpr bool kWidest = ALIGNED || FW == MOE_MX_E2M1;
    const int64_t widest = tiles(256, 256), last = (widest - 1) % 256 + 1;
    if (kWidest && last >= (widest <= 256 ? 168 : 128))
        launch_mx_tiled<FA, FW, kWidest ? 4 : 2, kWidest ? 4 : 2, ALIGNED>(a, s);
    else if (tiles(128, 128) >= 320) launch_mx_tiled<FA, FW, 2, 2, ALIGNED>(a, s);
    else if (tiles(64, 64) > 512) launch_mx_tiled<FA, FW, 1, 2, ALIGNED>(a, s);
    else launch_mx_tiled<FA, FW, 1, 1, ALIGNED>(a, s);
    return check_launch(name);
}

template <int FA, int FW>
int launch_mx_gemm(const MgArgs& a, hipStream_t s) {
    return (a.K / 32) % 4 == 0 && a.K >= 512 ? launch_mx_gemm<FA, FW, true>(a, s) : launch_mx_gemm<FA, FW, false>(a, s);
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
