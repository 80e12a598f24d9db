// Products grouped by expert on rows sorted by moe_dispatch, with their
// gradients: what a caller's own experts (or their backward pass) run between
// the sort of the tokens and the way back. Expert e's rows are
// [offsets[e], offsets[e] + counts[e]), w [E, N, D]:
//   moe_grouped_gemm        out[r, n]   = sum_d x[r, d] w[e, n, d]
//   moe_grouped_gemm_dgrad  d_x[r, d]   = sum_n d_out[r, n] w[e, n, d]
//   moe_grouped_gemm_wgrad  d_w[e, n, d] = sum_r d_out[r, n] x[r, d]     r over e's rows
//
// All three are one tiled kernel on the bf16 matrix unit (32 x 32 x 16, fp32
// accumulators). They differ in where an operand's contraction lies: along its
// rows in memory (x and w of the first, d_out of the second) or across them (w
// of the second, both of the third). The latter is staged in LDS as it lies in
// memory and turned on the way to the registers, by the LDS's transposing reads.
#include <type_traits>

#include "experts.hpp"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef float gg_f16v __attribute__((ext_vector_type(16)));

struct GgArgs {
    const uint8_t* a;       // the operand of the output's rows
    const uint8_t* b;       // the operand of its columns
    int64_t a_stride, b_stride, b_group;    // bytes; b_group: from expert to expert
    const int32_t* offsets;
    const int32_t* counts;
    int E;
    int64_t R;
    int blocks;             // of the output there are at most
    int M, N, K;            // output rows (weight gradient), output columns, contraction (else: the expert's rows)
    uint8_t* out;
    int64_t out_stride, out_group;          // bytes
    int out_vec;            // rows of out start at multiples of 16 bytes
};

constexpr int kGgElems = 64;        // contraction of a stage: 128 bytes of a row, a whole cache line
constexpr uint32_t kOutside = 0x80000000u;      // an offset past the descriptors' range: zeros arrive

// An operand whose rows hold the contraction: ROWS rows x 64 elements in LDS,
// the 8 chunks of a row permuted so that 16 consecutive rows' reads of one chunk
// spread over all banks.
template <int ROWS>
struct Along {
    static constexpr int kCopies = ROWS * 128 / 4096, kSize = ROWS * 128;
    const uint8_t* base;
    uint32_t off[kCopies];
    int chunk, k_bytes;
    __device__ __forceinline__ static int swizzle(int chunk, int row) { return chunk ^ (row & 7) ^ ((row >> 3) & 1); }
    __device__ __forceinline__ void init(const uint8_t* b, int64_t stride, int rows, int k, int wave, int lane) {
        base = b;
        const int r0 = 8 * wave + lane / 8;
        chunk = swizzle(lane % 8, r0);          // rows 32 apart have the same
        k_bytes = 2 * k;
#pragma unroll
        for (int q = 0; q < kCopies; ++q) off[q] = r0 + 32 * q < rows ? (uint32_t)((r0 + 32 * q) * stride + chunk * 16) : kOutside;
    }
    __device__ __forceinline__ void issue(uint32_t lds, int s, int q, int wave) const {
        lds_copy16(scalar_desc(base), __builtin_amdgcn_readfirstlane(lds + (4 * q + wave) * 1024),
                   s * 128 + chunk * 16 < k_bytes ? off[q] : kOutside, (uint32_t)__builtin_amdgcn_readfirstlane(s * 128));
    }
    // 8 elements of the contraction of row `row`: group g's of a step
    __device__ __forceinline__ static bf16x8 read(const uint8_t* at, int tile, int step, int lane) {
        const int row = 32 * tile + (lane & 31);
        return *reinterpret_cast<const bf16x8*>(at + row * 128 + 16 * swizzle(2 * step + (lane >> 5), row));
    }
};

// An operand whose contraction goes from row to row in memory: 64 rows x COLS
// columns in LDS. A transposing read hands a lane 4 rows of its column, while
// its 16 lanes fetch 4 rows x 32 bytes, and 32 lanes 4 rows x 64 bytes: those
// 64-byte pieces are permuted so that 4 consecutive rows' lie in different banks.
template <int COLS>
struct Across {
    static constexpr int kBytes = 2 * COLS, kChunks = kBytes / 16;
    static constexpr int kCopies = kGgElems * kBytes / 4096, kSize = kGgElems * kBytes;
    static constexpr bool kWhole = 256 % kChunks == 0;      // whole rows a copy of the 4 waves
    const uint8_t* base;
    int64_t stage;          // bytes from stage to stage
    uint32_t off[kCopies];
    int row[kWhole ? 1 : kCopies], k;
    __device__ __forceinline__ static int swizzle(int row) { return COLS % 128 == 0 ? row & 3 : COLS % 64 == 0 ? (row >> 1) & 1 : 0; }
    __device__ __forceinline__ int row_of(int q) const { return kWhole ? row[0] + 256 / kChunks * q : row[kWhole ? 0 : q]; }
    __device__ __forceinline__ void init(const uint8_t* b, int64_t stride, int cols, int contraction, int wave, int lane) {
        base = b;
        stage = kGgElems * stride;
        k = contraction;
#pragma unroll
        for (int q = 0; q < kCopies; ++q) {
            const int i = 64 * (4 * q + wave) + lane, r = i / kChunks, chunk = i % kChunks ^ (swizzle(r) << 2);
            if (!kWhole || q == 0) row[kWhole ? 0 : q] = r;
            off[q] = chunk * 8 < cols ? (uint32_t)(r * stride + chunk * 16) : kOutside;
        }
    }
    __device__ __forceinline__ void issue(uint32_t lds, int s, int q, int wave) const {
        lds_copy16(scalar_desc(base + s * stage), __builtin_amdgcn_readfirstlane(lds + (4 * q + wave) * 1024),
                   s * kGgElems + row_of(q) < k ? off[q] : kOutside, 0u);
    }
    __device__ __forceinline__ static bf16x8 read(const uint8_t* at, int tile, int step, int lane) {
        typedef __attribute__((address_space(3))) short4v lds4;
        const int r = 16 * step + 8 * (lane >> 5) + ((lane & 15) >> 2);
        const uint8_t* p = at + r * kBytes + ((tile ^ swizzle(r)) << 6) + 32 * ((lane >> 4) & 1) + 8 * (lane & 3);
        const short4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p));
        const short4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * kBytes));
        typedef short short8v __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(bf16x8, (short8v{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}));
    }
};

// ------------------------------------------------------------------ experts' rows
// What the maps hold of expert e: whatever that is, its rows stay inside [0, R).
__device__ __forceinline__ int gg_clamp(int v, int low, int high) { return v < low ? low : v < high ? v : high; }

// A block of the output and what it is computed from.
struct GgBlock {
    int e, row, rows, end;  // expert, its first row, its rows, the end of its padding rows
    int tile, tiles;        // the block among the expert's, the expert's blocks of rows
    int side, nt;           // the rows of each but the last, the expert's blocks of columns
    int tall;               // which of two shapes
};

__device__ __forceinline__ void gg_rows(const GgArgs& a, int e, GgBlock& b) {
    const int R = (int)a.R;
    b.e = e;
    b.row = gg_clamp(a.offsets[e], 0, R);
    b.end = gg_clamp(a.offsets[e + 1], b.row, R);
    b.rows = gg_clamp(a.counts[e], 0, b.end - b.row);
}

// XCD x (workgroups are dealt to the 8 round robin) gets a contiguous run of
// `total` blocks: which one this workgroup has, or -1.
__device__ __forceinline__ int xcd_run(int total) {
    const int x = blockIdx.x & 7, j = (int)(blockIdx.x >> 3), per = total >> 3, more = total & 7;
    return j < per + (x < more ? 1 : 0) ? x * per + (x < more ? x : more) + j : -1;
}

// The blocks of rows of an expert: of equal sides, as workgroups that go through
// the same weights at the same pace share them in the L2 (a small one runs ahead,
// out of its reach: 128 x 4096 x 1536, 264 rows each, forward 690 -> 628 us, input
// gradient 657 -> 577). Padding behind the last of up to half a block is that one's
// too; where there is more, whole blocks.
__device__ __forceinline__ int gg_split(GgBlock& g, int bm) {
    const int held = (g.rows + bm - 1) / bm, all = (g.end - g.row + bm - 1 - bm / 2) / bm;
    g.tiles = g.end == g.row ? 0 : held > all ? held : all > 1 ? all : 1;
    g.side = held > 1 && held == g.tiles ? ((g.rows - 1) / held + 16) & ~15 : bm;
    return held;
}

// Blocks of bm x bn or, where an expert's rows fill fewer blocks of them and all its
// blocks are less work, tall ones (TALL: 320 x 192, 15 tiles a wave against 16).
template <int BM, int BN, bool TALL>
__device__ __forceinline__ void gg_shape(int N, GgBlock& g) {
    const int held = gg_split(g, BM);
    g.nt = (N + BN - 1) / BN;
    g.tall = 0;
    if constexpr (TALL) {
        GgBlock t = g;
        t.nt = (N + 191) / 192;
        t.tall = 1;
        if (gg_split(t, 320) < held && 15 * t.tiles * t.nt < 16 * g.tiles * g.nt) g = t;
    }
}

// The expert and block of this workgroup: experts in order, each with its blocks.
// Every thread counts a few experts'; at most a.blocks in all (more only where the
// maps are wrong).
template <int BM, int BN, bool TALL>
__device__ __forceinline__ bool gg_find(const GgArgs& a, GgBlock& out, uint8_t* lds) {
    int* s_sum = reinterpret_cast<int*>(lds);
    GgBlock& s_out = *reinterpret_cast<GgBlock*>(lds + 16);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (a.E + 255) / 256, e0 = tid * per;
    int mine = 0;
    for (int e = e0; e < e0 + per && e < a.E; ++e) {
        GgBlock g;
        gg_rows(a, e, g);
        gg_shape<BM, BN, TALL>(a.N, g);
        mine += g.tiles * g.nt;
    }
    mine = mine < a.blocks ? mine : a.blocks;       // (a.blocks <= 2^24: a wave's sum stays in 31 bits)
    const int upto = wave_inclusive_scan(mine);
    if (lane == 63) s_sum[wave] = upto;
    if (tid == 0) s_out.e = -1;
    __syncthreads();
    int64_t before = upto - mine, total = 0;
    for (int w = 0; w < 4; ++w) {
        if (w < wave) before += s_sum[w];
        total += s_sum[w];
    }
    const int id = xcd_run((int)(total < a.blocks ? total : a.blocks));
    if (id < 0) return false;
    if (id >= before && id < before + mine) {
        for (int e = e0; e < e0 + per && e < a.E; ++e) {
            GgBlock g;
            gg_rows(a, e, g);
            gg_shape<BM, BN, TALL>(a.N, g);
            g.tile = (int)(id - before);
            if (id >= before && id < before + g.tiles * g.nt) s_out = g;
            before += g.tiles * g.nt;
        }
    }
    __syncthreads();
    out.e = __builtin_amdgcn_readfirstlane(s_out.e);
    out.row = __builtin_amdgcn_readfirstlane(s_out.row);
    out.rows = __builtin_amdgcn_readfirstlane(s_out.rows);
    out.end = __builtin_amdgcn_readfirstlane(s_out.end);
    out.tile = __builtin_amdgcn_readfirstlane(s_out.tile);
    out.tiles = __builtin_amdgcn_readfirstlane(s_out.tiles);
    out.side = __builtin_amdgcn_readfirstlane(s_out.side);
    out.nt = __builtin_amdgcn_readfirstlane(s_out.nt);
    out.tall = __builtin_amdgcn_readfirstlane(s_out.tall);
    __syncthreads();        // the block's operands come there
    return out.e >= 0;
}

// ------------------------------------------------------------------ output
// 32 rows x NT tiles of 32 columns of a wave's block, bf16, turned in the wave's own
// part of the LDS: a lane holds 4 consecutive columns of one row at a time, and whole
// 16-byte pieces of the rows are stored. Of `left` rows, those from `live` on are
// zeros. ADD: added to what the output holds, in fp32 (in the LDS too), rounded once.
template <int NT, bool ADD>
constexpr int gg_row_bytes() { return 32 * NT * (ADD ? 4 : 2) + 16; }

template <int NT, bool ADD>
__device__ __forceinline__ void gg_store(uint8_t* out, int64_t stride, bool vec, uint8_t* slab, const gg_f16v (&acc)[NT],
                                         int live, int left, int cols, int lane) {
    constexpr int kRow = gg_row_bytes<NT, ADD>(), kPieces = 4 * NT, kCount = kPieces / 2, kBatch = kCount < 8 ? kCount : kCount / 2;
    static_assert(kCount % kBatch == 0, "whole batches");
    const int r = lane & 31, g = lane >> 5;
    const bool zero = r >= live;
    wave_lds_sync();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = 32 * n + 8 * q + 4 * g;
            const gg_f16v& a = acc[n];
            const float v0 = zero ? 0.0f : a[4 * q], v1 = zero ? 0.0f : a[4 * q + 1];
            const float v2 = zero ? 0.0f : a[4 * q + 2], v3 = zero ? 0.0f : a[4 * q + 3];
            if constexpr (ADD) *reinterpret_cast<floatx4*>(slab + r * kRow + c * 4) = floatx4{v0, v1, v2, v3};
            else *reinterpret_cast<uint2*>(slab + r * kRow + c * 2) = make_uint2(bf16x2_pack(v0, v1), bf16x2_pack(v2, v3));
        }
    wave_lds_sync();
    // piece lane + 64 j of the rows' in order: where 64 are whole rows, from j to j the same rows further down
    constexpr bool kEven = 64 % kPieces == 0;
    constexpr int kRowsPer = kEven ? 64 / kPieces : 0;
    const int lane_row = lane / kPieces, lane_col = lane % kPieces * 8;
    const auto row = [&](int j) { return kEven ? lane_row + j * kRowsPer : (lane + 64 * j) / kPieces; };
    const auto col = [&](int j) { return kEven ? lane_col : (lane + 64 * j) % kPieces * 8; };
    const uint8_t* src0 = slab + lane_row * kRow + lane_col * (ADD ? 4 : 2);
    uint8_t* dst0 = out + lane_row * stride + lane_col * 2;
    const auto src = [&](int j) { return kEven ? src0 + j * kRowsPer * kRow : slab + row(j) * kRow + col(j) * (ADD ? 4 : 2); };
    const auto dst = [&](int j) { return kEven ? dst0 + j * kRowsPer * stride : out + row(j) * stride + col(j) * 2; };
    // a piece of the output: what LDS holds, or that and the output's own
    const auto piece = [](const uint8_t* p, u32x4 old) {
        if constexpr (!ADD) {
            return *reinterpret_cast<const u32x4*>(p);
        } else {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lo = reinterpret_cast<const float*>(p)[2 * i], hi = reinterpret_cast<const float*>(p)[2 * i + 1];
                o[i] = bf16x2_pack(__fadd_rn(lo, bf16_to_f32(old[i] & 0xFFFFu)), __fadd_rn(hi, __uint_as_float(old[i] & 0xFFFF0000u)));
            }
            return o;
        }
    };
    if (vec && left >= 32 && cols >= 32 * NT) {
#pragma unroll
        for (int j0 = 0; j0 < kCount; j0 += kBatch) {
            u32x4 v[kBatch] = {};
            if constexpr (ADD) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j) v[j] = *reinterpret_cast<const u32x4*>(dst(j0 + j));
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) v[j] = piece(src(j0 + j), v[j]);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) __builtin_nontemporal_store(v[j], reinterpret_cast<u32x4*>(dst(j0 + j)));
        }
        return;
    }
#pragma unroll 1
    for (int j = 0; j < kCount; ++j) {
        const int c = col(j);
        if (row(j) >= left || c >= cols) continue;
        if (vec) {          // (columns come in eights: whole pieces)
            u32x4 old = {};
            if constexpr (ADD) old = *reinterpret_cast<const u32x4*>(dst(j));
            __builtin_nontemporal_store(piece(src(j), old), reinterpret_cast<u32x4*>(dst(j)));
        } else if constexpr (!ADD) {        // rows at any stride; d_w's are contiguous
            for (int k = 0; k < 8; ++k) reinterpret_cast<uint16_t*>(dst(j))[k] = reinterpret_cast<const uint16_t*>(src(j))[k];
        }
    }
}

// The same of fp32, straight from the accumulators: there a lane holds one
// column of 4 consecutive rows at a time, so that 32 lanes store a row's whole cache
// line (or part of it, at any stride). Weight gradient of 128 experts x 4096 x 1536,
// 256 rows each: 892 -> 814 us. With ADD each step of 4 rows reads, waits, adds and
// stores in turn, and there is one block a CU to do it: 2529 us, where the bytes alone
// are 1.4 ms.
template <int NT, bool ADD>
__device__ __forceinline__ void gg_store32(uint8_t* out, int64_t stride, const gg_f16v (&acc)[NT], int live, int left, int cols, int lane) {
    const int c = lane & 31, g = lane >> 5;
    uint8_t* at = out + 4 * g * stride + 4 * c;
    if (live >= 32 && cols >= 32 * NT) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float* row = reinterpret_cast<float*>(at + (8 * (i / 4) + i % 4) * stride);
            float v[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) v[n] = ADD ? row[32 * n] : 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n) __builtin_nontemporal_store(ADD ? __fadd_rn(acc[n][i], v[n]) : acc[n][i], row + 32 * n);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = 8 * (i / 4) + i % 4 + 4 * g;
        float* row = reinterpret_cast<float*>(at + (8 * (i / 4) + i % 4) * stride);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (r >= left || 32 * n + c >= cols) continue;
            const float v = r < live ? acc[n][i] : 0.0f;
            __builtin_nontemporal_store(ADD ? __fadd_rn(v, row[32 * n]) : v, row + 32 * n);
        }
    }
}

// ------------------------------------------------------------------ the kernel
// 4 waves, WM along the output's rows; a wave has MW x NW tiles of 32 x 32, its
// tiles' rows dealt round the waves, so that a block of few rows is few tiles of
// every wave's.
//
// What bounds it: 128 experts x 4096 x 1536, 4096 tokens top-8, in 495 us forward is
// 4.0 TB/s of the 1.98 GB that have to move (a large copy reaches 4.8) at 0.83
// PFLOP/s; 8 experts of 4096 rows each in 365 to 370, 1.12 PFLOP/s (a large library product
// 1.45). A stage's copies take 0.6 to 1 us to arrive, and the bytes in flight are what
// LDS holds: hence large blocks, one a CU, and a ring that takes all of it. The 64
// rows of 8 tokens, 64 x 1536 x 2048, read their experts' 254 MB of weights in 47 us,
// 5.4 TB/s.
enum GgKind { kGgRows, kGgRowsT, kGgWeight };       // forward, input gradient, weight gradient

template <int KIND, int WM, int MW, int NW, bool F32, bool ADD>
struct GgShape {
    static constexpr int kWN = 4 / WM, kBM = 32 * WM * MW, kBN = 32 * kWN * NW;
    using A = std::conditional_t<KIND == kGgWeight, Across<kBM>, Along<kBM>>;
    using B = std::conditional_t<KIND == kGgRows, Along<kBN>, Across<kBN>>;
    static constexpr int kSlab = F32 ? 0 : 32 * gg_row_bytes<NW, ADD>();
    static constexpr bool kTall = KIND != kGgWeight && MW * NW == 16;     // beside tall blocks
    static constexpr int kPerCu = MW * NW >= 12 ? 1 : 2, kLds = 160 * 1024 / kPerCu;
    // A ring of stages for a block of LIVE row tiles a wave: what such a block does not need makes room for more of them.
    template <int LIVE>
    struct Ring {
        static constexpr int kCopiesA = KIND == kGgWeight ? A::kCopies : WM * LIVE, kAll = kCopiesA + B::kCopies;
        static constexpr int kSizeA = 4096 * kCopiesA, kStage = kSizeA + B::kSize;
        static constexpr int kFit = kLds / kStage, kRing = kFit < 6 ? kFit : 6;
        static_assert(kRing >= 2 && kRing * kAll < 64, "ring of stages");
    };
    static_assert(4 * kSlab <= kLds, "the waves' slabs");
};

// LEAST: no block has fewer row tiles a wave than that (it may have fewer that hold rows).
template <int KIND, int WM, int MW, int NW, bool F32, bool ADD, int LEAST>
__device__ __forceinline__ void gg_block(const GgArgs& a, const GgBlock& b, uint8_t* lds) {
    using S = GgShape<KIND, WM, MW, NW, F32, ADD>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / S::kWN, wn = wave % S::kWN, nt = b.nt;
    // groups of 4 blocks of rows, column by column: what neighbours share stays in the XCD's L2
    const int gm0 = b.tile / (4 * nt) * 4, gh = b.tiles - gm0 < 4 ? b.tiles - gm0 : 4, in = b.tile - gm0 * nt;
    const int mt = gm0 + in % gh, m0 = mt * b.side, n0 = (in / gh) * S::kBN;
    // rows of the block that are computed, and that are written (the last block has all that are left); contraction
    const int left = KIND == kGgWeight ? a.M - m0 : mt + 1 < b.tiles ? b.side : b.end - b.row - m0;
    const int live = KIND == kGgWeight ? left : b.rows - m0 < left ? b.rows - m0 : left;
    const int k = KIND == kGgWeight ? b.rows : live > 0 ? a.K : 0, stages = (k + kGgElems - 1) / kGgElems;
    if (ADD && k == 0) return;

    typename S::A ca;
    typename S::B cb;
    const uint32_t lds0 = lds_addr(lds);
    if (stages > 0) {
        if constexpr (KIND == kGgWeight) {
            ca.init(a.a + b.row * a.a_stride + 2 * (int64_t)m0, a.a_stride, live, k, wave, lane);
            cb.init(a.b + b.row * a.b_stride + 2 * (int64_t)n0, a.b_stride, a.N - n0, k, wave, lane);
        } else {
            const uint8_t* w = a.b + b.e * a.b_group;
            ca.init(a.a + (b.row + (int64_t)m0) * a.a_stride, a.a_stride, live, k, wave, lane);
            if constexpr (KIND == kGgRows) cb.init(w + n0 * a.b_stride, a.b_stride, a.N - n0, k, wave, lane);
            else cb.init(w + 2 * (int64_t)n0, a.b_stride, a.N - n0, k, wave, lane);
        }
    }
    struct Operands {
        bf16x8 a[MW], b[NW];
    };
    constexpr int kSlots = MW * NW, kReads = 2 * (MW + NW), kFree = kSlots / 4, kCopySlots = 2 * kSlots - kFree;

    // The block, of which LIVE row tiles a wave or fewer hold rows.
    //
    // A ring of stages, a stage four steps of 16. Its operands are read in two
    // bursts around its beginning, steps 0 and 1 during the last step of the stage
    // before, 2 and 3 during its first: the buffer is free soon after (the first
    // barrier; the copies of stage s + kRing go into it, spread over the MFMAs that
    // follow), and the next one is not needed before the last step (the second
    // barrier, in front of which every wave waits for its own copies). So a copy
    // has half a stage more to arrive than the ring has stages.
    auto compute = [&](auto tiles) __attribute__((always_inline)) {
        constexpr int LIVE = decltype(tiles)::value;
        using R = typename S::template Ring<LIVE>;
        constexpr int kAll = R::kAll;
        // Rows whose length is a multiple of some KB meet in few memory channels at one place along them: forward, where both
        // operands are read along their rows, blocks begin at different stages and go round, by expert and columns (us; 64 x
        // 1536 x 2048: 8 tokens' rows 53 to 57 -> 47, 16 rows an expert 78 to 84 -> 71, 128 rows 90 -> 86; 128 x 4096 x 1536, 256
        // rows each 460 -> 445, routed 486 to 497 -> 486). The gradients gain nothing by it.
        const int start = KIND == kGgRows && stages > 0 ? (int)((unsigned)(b.e * nt + n0 / S::kBN) % (unsigned)stages) : 0;
        auto copy = [&](int s, int q0, int q1) __attribute__((always_inline)) {        // copies [q0, q1) of stage s
            const uint32_t at = lds0 + (s % R::kRing) * R::kStage;
            if (KIND == kGgRows && s < stages) {
                s += start;
                if (s >= stages) s -= stages;
            }
#pragma unroll
            for (int q = q0; q < q1; ++q) {
                if (q < R::kCopiesA) ca.issue(at, s, q, wave);
                else cb.issue(at + R::kSizeA, s, q - R::kCopiesA, wave);
            }
        };
        if (stages > 0) {
#pragma unroll
            for (int s = 0; s < R::kRing; ++s) copy(s, 0, kAll);
        }
        gg_f16v acc[LIVE][NW];
#pragma unroll
        for (int m = 0; m < LIVE; ++m)
#pragma unroll
            for (int n = 0; n < NW; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.0f;
        if (stages > 0) {
            Operands o0, o1, o2, o3;
            auto read = [&](int s, int step, Operands& o, int i) __attribute__((always_inline)) {  // operand i: the columns', then the rows'
                const uint8_t* at = lds + (s % R::kRing) * R::kStage;
                if (i < NW) o.b[i] = S::B::read(at + R::kSizeA, wn * NW + i, step, lane);
                else if (i < NW + LIVE) o.a[i - NW] = S::A::read(at, wm + WM * (i - NW), step, lane);
            };
            auto mfma = [&](const Operands& o, int i) __attribute__((always_inline)) {             // MFMA i of a step
                if (i / NW < LIVE)
                    acc[i / NW][i % NW] = F32 ? __builtin_amdgcn_mfma_f32_32x32x16_bf16(o.a[i / NW], o.b[i % NW], acc[i / NW][i % NW], 0, 0, 0)
                                              : __builtin_amdgcn_mfma_f32_32x32x16_bf16(o.b[i % NW], o.a[i / NW], acc[i / NW][i % NW], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            };
            __builtin_amdgcn_s_waitcnt(vmcnt_at_most((R::kRing - 1) * kAll));
            asm volatile("s_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kReads; ++i) read(0, i < kReads / 2 ? 0 : 1, i < kReads / 2 ? o0 : o1, i % (kReads / 2));
            for (int s = 0; s < stages; ++s) {
#pragma unroll
                for (int i = 0; i < kSlots; ++i) {
#pragma unroll
                    for (int j = i * kReads / kSlots; j < (i + 1) * kReads / kSlots; ++j)
                        read(s, j < kReads / 2 ? 2 : 3, j < kReads / 2 ? o2 : o3, j % (kReads / 2));
                    mfma(o0, i);
                }
#pragma unroll
                for (int i = 0; i < 2 * kSlots; ++i) {
                    if (i == kFree) {
                        __builtin_amdgcn_s_waitcnt(lgkmcnt_zero());
                        asm volatile("s_barrier" ::: "memory");
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if (i >= kFree) copy(s + R::kRing, (i - kFree) * kAll / kCopySlots, (i - kFree + 1) * kAll / kCopySlots);
                    mfma(i < kSlots ? o1 : o2, i % kSlots);
                }
                __builtin_amdgcn_s_waitcnt(vmcnt_at_most((R::kRing - 1) * kAll));
                asm volatile("s_barrier" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < kSlots; ++i) {
#pragma unroll
                    for (int j = i * kReads / kSlots; j < (i + 1) * kReads / kSlots; ++j)
                        read(s + 1, j < kReads / 2 ? 0 : 1, j < kReads / 2 ? o0 : o1, j % (kReads / 2));
                    mfma(o3, i);
                }
            }
            // the copies of the stages behind the last still write (zeros) to the LDS
            __builtin_amdgcn_s_waitcnt(vmcnt_at_most(0) & lgkmcnt_zero());
            __syncthreads();
        }
        uint8_t* slab = lds + wave * S::kSlab;
        const int c0 = n0 + 32 * NW * wn;
#pragma unroll
        for (int m = 0; m < LIVE; ++m) {
            const int r0 = 32 * (wm + WM * m);
            if (r0 >= left || c0 >= a.N) continue;
            uint8_t* out = a.out + (KIND == kGgWeight ? b.e * a.out_group + (m0 + r0) * a.out_stride
                                                      : (b.row + (int64_t)m0 + r0) * a.out_stride);
            out += (int64_t)c0 * (F32 ? 4 : 2);
            if constexpr (F32) gg_store32<NW, ADD>(out, a.out_stride, acc[m], live - r0, left - r0, a.N - c0, lane);
            else gg_store<NW, ADD>(out, a.out_stride, a.out_vec, slab, acc[m], live - r0, left - r0, a.N - c0, lane);
            __builtin_amdgcn_sched_barrier(0);
        }
        // rows of padding behind those tiles: whole pieces of 16 bytes (N % 8 == 0) where rows start at such
        if constexpr (KIND != kGgWeight) {
            constexpr int kEs = F32 ? 4 : 2, kPieces = 2 * NW * kEs;
            for (int i = lane; i < (left - 32 * WM * LIVE) * kPieces; i += 64) {
                const int r = 32 * WM * LIVE + i / kPieces, c = c0 * kEs + i % kPieces * 16;
                if (r % WM != wm || c >= a.N * kEs) continue;
                uint8_t* out = a.out + (b.row + (int64_t)m0 + r) * a.out_stride + c;
                if (a.out_vec) __builtin_nontemporal_store(u32x4{}, reinterpret_cast<u32x4*>(out));
                else
                    for (int k = 0; k < 16 / kEs; ++k) {
                        if constexpr (F32) reinterpret_cast<float*>(out)[k] = 0.0f;
                        else reinterpret_cast<uint16_t*>(out)[k] = 0;
                    }
            }
        }
    };
    const int tiles = (live + 32 * WM - 1) / (32 * WM);
    if (MW >= 5 && (LEAST >= 5 || tiles >= 5)) compute(std::integral_constant<int, (MW >= 5 ? 5 : 1)>());
    else if constexpr (LEAST < 5) {
        if (MW >= 4 && tiles >= 4) compute(std::integral_constant<int, (MW >= 4 ? 4 : 1)>());
        else if (MW >= 3 && tiles >= 3) compute(std::integral_constant<int, (MW >= 3 ? 3 : 1)>());
        else if (MW >= 2 && tiles >= 2) compute(std::integral_constant<int, (MW >= 2 ? 2 : 1)>());
        else compute(std::integral_constant<int, 1>());
    }
}

template <int KIND, int WM, int MW, int NW, bool F32, bool ADD>
__global__ void __launch_bounds__(256, (GgShape<KIND, WM, MW, NW, F32, ADD>::kPerCu)) grouped_gemm_kernel(GgArgs a) {
    using S = GgShape<KIND, WM, MW, NW, F32, ADD>;
    __shared__ __align__(16) uint8_t lds[S::kLds];
    GgBlock b;
    if constexpr (KIND == kGgWeight) {
        b.tiles = (a.M + S::kBM - 1) / S::kBM;
        b.nt = (a.N + S::kBN - 1) / S::kBN;
        b.side = S::kBM;
        const int id = xcd_run(a.blocks), e = id / (b.tiles * b.nt);
        if (id < 0) return;
        gg_rows(a, e, b);
        b.tile = id - e * (b.tiles * b.nt);
    } else {
        if (!gg_find<S::kBM, S::kBN, S::kTall>(a, b, lds)) return;
        if constexpr (S::kTall)
            if (b.tall) return gg_block<KIND, 2, 5, 3, F32, ADD, 5>(a, b, lds);
    }
    gg_block<KIND, WM, MW, NW, F32, ADD, 1>(a, b, lds);
}

// ------------------------------------------------------------------ host side
template <int KIND, int WM, int MW, int NW, bool F32, bool ADD>
int launch_grouped(GgArgs a, hipStream_t s, const char* name) {
    using S = GgShape<KIND, WM, MW, NW, F32, ADD>;
    const int64_t nt = (a.N + S::kBN - 1) / S::kBN;
    const int64_t row_blocks = a.R / S::kBM + (a.R < a.E ? a.R : a.E);      // whole blocks, and each expert's last
    int64_t blocks = KIND == kGgWeight ? (int64_t)a.E * ((a.M + S::kBM - 1) / S::kBM) * nt : row_blocks * nt;
    if (S::kTall) blocks += blocks / 15;        // tall ones where they are fewer, or up to so many more
    const int64_t grid = (blocks + 7) / 8 * 8;
    if (!launch_fits(grid, 256)) return fail(MOE_EUNSUPPORTED, "%s: too many output tiles", name);
    a.blocks = (int)blocks;
    hipLaunchKernelGGL((grouped_gemm_kernel<KIND, WM, MW, NW, F32, ADD>), dim3((unsigned)grid), dim3(256), 0, s, a);
    return check_launch(name);
}

template <int KIND, int WM, int MW, int NW>
int launch_grouped(const GgArgs& a, bool f32, bool add, hipStream_t s, const char* name) {
    if constexpr (KIND == kGgWeight) {
        if (add) return f32 ? launch_grouped<KIND, WM, MW, NW, true, true>(a, s, name) : launch_grouped<KIND, WM, MW, NW, false, true>(a, s, name);
    }
    return f32 ? launch_grouped<KIND, WM, MW, NW, true, false>(a, s, name) : launch_grouped<KIND, WM, MW, NW, false, false>(a, s, name);
}

// Sizes of the three calls.
static int gg_sizes(int64_t rows_max, int E, int N, int D, int dtype, const char* name) {
    if (rows_max < 0 || rows_max > 0x7FFFFFFF || E < 1 || E > MOE_MAX_EXPERTS || N < 0 || D < 0)
        return fail(MOE_EINVAL, "%s: rows_max=%lld E=%d N=%d D=%d out of range", name, (long long)rows_max, E, N, D);
    if (dtype != MOE_BF16 && dtype != MOE_F32)
        return fail(MOE_EINVAL, "%s: dtype %d is neither MOE_BF16 nor MOE_F32", name, dtype);
    if (N % 8 || D % 8 || N > MOE_MAX_GROUPED || D > MOE_MAX_GROUPED)
        return fail(MOE_EUNSUPPORTED, "%s: N=%d and D=%d must be multiples of 8 up to %d", name, N, D, MOE_MAX_GROUPED);
    if (rows_max > MOE_MAX_ROWS)        // a block, or a ring of stages, behind the last row stays in 31 bits
        return fail(MOE_EUNSUPPORTED, "%s: rows_max=%lld is more than %d", name, (long long)rows_max, MOE_MAX_ROWS);
    return MOE_OK;
}

// Whether the last round of blocks, one a CU, is 0.8 full or one of many.
static bool gg_filled(int64_t blocks) { return blocks >= 1024 || 10 * blocks >= 8 * ((blocks + 255) / 256 * 256); }

// The block's rows for the forward product and the input's gradient. Wide blocks
// read less per product, from the L2 and of the weights; but a CU without one
// idles, and where an expert has few rows a block is mostly empty (its empty row
// tiles are not computed). rows_max counts padding and routes that went elsewhere:
// the experts' rows are only guessed from it. us, blocks of 256 x 256 (with tall ones),
// 128 x 128 and 32 x 128, forward and input gradient, every expert of the same rows:
//   E x N x D        rows each
//   128 x 4096 x 1536  256   450 422   567 518   1080 977     8 x 4096 x 1536   4096   370 348   439 422   876 850
//   128 x 4096 x 1536  128   336 311   385 360    626 554   128 x 4096 x 1536     32   289 287   297 304   295 304
//    64 x 1536 x 2048  128    92  86    85  89    143 150    64 x 1536 x 2048     64    81  76    76  79    95  97
//    64 x 1536 x 2048   16    77  74    72  75     72  75     8 x 1536 x 2048    256    40  35    19  18    29  31
//     8 x 1536 x 2048   64    22  21    15  16     13  12     1 x 4096 x 4096   1024    72  79    39  40    65  72
//     1 x 4096 x 4096  256    71  78    31  32     22  23   128 x 4096 x 1536      4   129 142   115 130   113 128
// (the last in the mean, skewed). Rows of fp32 take 0 to 6% more, in the same order. 256
// rows in the mean of a routing, 128 x 4096 x 1536: 496 485, 614 586, 1133 1040. Not seen
// by the rule: how much of rows_max is padding (512 routes over 128 experts in tiles of
// 128 rows count as 16768 rows, and take the wide blocks: 4 rows each, the last line).
static int gg_rows_blocks(int64_t rows_max, int E, int cols) {
    const auto blocks = [&](int64_t side) {         // about: half a block of rows is lost an expert
        const int64_t rows = rows_max / side + (rows_max < E ? rows_max : E) / 2, least = rows_max < E ? rows_max : E;
        return (rows > least ? rows : least) * ((cols + side - 1) / side);
    };
    const int64_t wide = blocks(256);
    if (rows_max >= 32 * (int64_t)E && wide >= 200 && (wide >= 448 || (rows_max >= 96 * (int64_t)E && gg_filled(wide)))) return 256;
    if (rows_max >= 32 * (int64_t)E && blocks(128) >= 150) return 128;
    return 32;
}

// Row strides of the operands: at least the row, whole 16-byte pieces, and a block's rows within 31 bits.
static bool gg_bad_stride(int64_t stride, int cols) { return stride < cols || stride % 8 || stride > (1 << 21); }

static int gg_maps(const int32_t* offsets, const int32_t* counts, const char* name) {
    if (!offsets || !counts) return fail(MOE_EINVAL, "%s: NULL pointer", name);
    if (!aligned16(offsets) || !aligned16(counts)) return fail(MOE_EINVAL, "%s: pointers must be 16-byte aligned", name);
    return MOE_OK;
}

// Forward and input gradient: rows [rows_max, in_cols] to rows [rows_max, out_cols].
static int gg_rows_call(const uint16_t* x, int64_t x_row_stride, const uint16_t* w, const int32_t* offsets, const int32_t* counts,
                        int64_t rows_max, int E, int N, int D, bool input_grad, void* out, int64_t out_row_stride, int out_dtype,
                        void* stream, const char* name) {
    int rc = gg_sizes(rows_max, E, N, D, out_dtype, name);
    const int in_cols = input_grad ? N : D, out_cols = input_grad ? D : N;
    if (rc != MOE_OK || rows_max == 0 || out_cols == 0) return rc;
    rc = gg_maps(offsets, counts, name);
    if (rc != MOE_OK) return rc;
    if (!out || (in_cols && (!x || !w))) return fail(MOE_EINVAL, "%s: NULL pointer", name);
    if (!aligned16(x) || !aligned16(w) || !aligned16(out)) return fail(MOE_EINVAL, "%s: pointers must be 16-byte aligned", name);
    if ((in_cols && gg_bad_stride(x_row_stride, in_cols)) || out_row_stride < out_cols)
        return fail(MOE_EINVAL, "%s: row strides must be >= the rows (the input's a multiple of 8, at most %d)", name, 1 << 21);
    GgArgs a{};
    a.a = (const uint8_t*)x; a.a_stride = 2 * x_row_stride;
    a.b = (const uint8_t*)w; a.b_stride = 2 * (int64_t)D; a.b_group = 2 * (int64_t)N * D;
    a.offsets = offsets; a.counts = counts; a.E = E; a.R = rows_max; a.N = out_cols; a.K = in_cols;
    const bool f32 = out_dtype == MOE_F32;
    a.out = (uint8_t*)out; a.out_stride = out_row_stride * (f32 ? 4 : 2); a.out_vec = a.out_stride % 16 == 0;
    hipStream_t s = (hipStream_t)stream;
    switch (gg_rows_blocks(rows_max, E, out_cols)) {
        case 256: return input_grad ? launch_grouped<kGgRowsT, 2, 4, 4>(a, f32, false, s, name) : launch_grouped<kGgRows, 2, 4, 4>(a, f32, false, s, name);
        case 128: return input_grad ? launch_grouped<kGgRowsT, 2, 2, 2>(a, f32, false, s, name) : launch_grouped<kGgRows, 2, 2, 2>(a, f32, false, s, name);
        default: return input_grad ? launch_grouped<kGgRowsT, 1, 1, 1>(a, f32, false, s, name) : launch_grouped<kGgRows, 1, 1, 1>(a, f32, false, s, name);
    }
}

}  // namespace moe

extern "C" int moe_grouped_gemm(const uint16_t* x, int64_t x_row_stride, const uint16_t* w, const int32_t* expert_offsets,
                                const int32_t* expert_counts, int64_t rows_max, int E, int N, int D, void* out,
                                int64_t out_row_stride, int out_dtype, void* stream) {
    return moe::gg_rows_call(x, x_row_stride, w, expert_offsets, expert_counts, rows_max, E, N, D, false, out, out_row_stride,
                             out_dtype, stream, "moe_grouped_gemm");
}

extern "C" int moe_grouped_gemm_dgrad(const uint16_t* d_out, int64_t d_out_row_stride, const uint16_t* w,
                                      const int32_t* expert_offsets, const int32_t* expert_counts, int64_t rows_max, int E, int N,
                                      int D, void* d_x, int64_t d_x_row_stride, int d_x_dtype, void* stream) {
    return moe::gg_rows_call(d_out, d_out_row_stride, w, expert_offsets, expert_counts, rows_max, E, N, D, true, d_x,
                             d_x_row_stride, d_x_dtype, stream, "moe_grouped_gemm_dgrad");
}

extern "C" int moe_grouped_gemm_wgrad(const uint16_t* d_out, int64_t d_out_row_stride, const uint16_t* x, int64_t x_row_stride,
                                      const int32_t* expert_offsets, const int32_t* expert_counts, int64_t rows_max, int E, int N,
                                      int D, int accumulate, void* d_w, int d_w_dtype, void* stream) {
    using namespace moe;
    const char* name = "moe_grouped_gemm_wgrad";
    int rc = gg_sizes(rows_max, E, N, D, d_w_dtype, name);
    if (rc != MOE_OK || N == 0 || D == 0) return rc;
    rc = gg_maps(expert_offsets, expert_counts, name);
    if (rc != MOE_OK) return rc;
    if (!d_w || (rows_max && (!d_out || !x))) return fail(MOE_EINVAL, "%s: NULL pointer", name);
    if (!aligned16(d_out) || !aligned16(x) || !aligned16(d_w)) return fail(MOE_EINVAL, "%s: pointers must be 16-byte aligned", name);
    if (gg_bad_stride(d_out_row_stride, N) || gg_bad_stride(x_row_stride, D))
        return fail(MOE_EINVAL, "%s: row strides must be >= the rows and multiples of 8, at most %d", name, 1 << 21);
    const bool f32 = d_w_dtype == MOE_F32;
    GgArgs a{};
    a.a = (const uint8_t*)d_out; a.a_stride = 2 * d_out_row_stride;
    a.b = (const uint8_t*)x; a.b_stride = 2 * x_row_stride;
    a.offsets = expert_offsets; a.counts = expert_counts; a.E = E; a.R = rows_max; a.M = N; a.N = D;
    a.out = (uint8_t*)d_w; a.out_stride = (int64_t)D * (f32 ? 4 : 2); a.out_group = a.out_stride * N; a.out_vec = a.out_stride % 16 == 0;
    // us, blocks of 256 x 256 and 128 x 128, bf16 d_w and fp32:
    //   128 x 4096 x 1536, rows each 256   672 762   814 1033      64 x 1536 x 2048, 128   121 122   148 145
    //                                128   512 590   637  695                         64   104 102   139 122
    //                                 32   389 388   584  569                         16   102  99   133 127
    //                  4 in the mean, skewed 328 310 591  564       8 x 1536 x 2048, 256    27  23    30  26
    //     8 x 4096 x 1536,          4096   345 443   354  455       1 x 4096 x 4096, 1024   35  40    40  41
    // Accumulating: 128 x 4096 x 1536, 256 997 944 2529 2538, 32 784 696 2372 2385; 8 x 4096 x 1536, 4096 368 453 449 496 (the
    // rule has no term for it, though bf16 sums onto many experts' weights are quicker in the smaller blocks)
    // (a block of few rows is its output alone, which the smaller ones write beside another's reads; not so in long runs)
    const int64_t wide = (int64_t)E * ((N + 255) / 256) * ((D + 255) / 256);
    if (rows_max >= (wide >= 4096 ? 96 : 192) * (int64_t)E && wide >= 200 && gg_filled(wide))
        return launch_grouped<kGgWeight, 2, 4, 4>(a, f32, accumulate != 0, (hipStream_t)stream, name);
    return launch_grouped<kGgWeight, 2, 2, 2>(a, f32, accumulate != 0, (hipStream_t)stream, name);
}
