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
    u32x4 rsrc;
    uint32_t off[kCopies];
    int chunk, k_bytes;
    __device__ __forceinline__ static int swizzle(int chunk, int row) { return chunk ^ (row & 7) ^ ((row >> 3) & 1); }
    __device__ __forceinline__ void init(const uint8_t* base, int64_t stride, int rows, int k, int wave, int lane) {
        rsrc = buffer_desc(base);
        const int r0 = 8 * wave + lane / 8;
        chunk = swizzle(lane % 8, r0);          // rows 32 apart have the same
        k_bytes = 2 * k;
#pragma unroll
        for (int q = 0; q < kCopies; ++q) off[q] = r0 + 32 * q < rows ? (uint32_t)((r0 + 32 * q) * stride + chunk * 16) : kOutside;
    }
    __device__ __forceinline__ void issue(uint32_t lds, int s, int q, int wave) const {
        lds_copy16(rsrc, __builtin_amdgcn_readfirstlane(lds + (4 * q + wave) * 1024),
                   s * 128 + chunk * 16 < k_bytes ? off[q] : kOutside, (uint32_t)(s * 128));
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
    static constexpr int kBytes = 2 * COLS, kChunks = kBytes / 16, kRowsPer = 64 / kChunks;
    static constexpr int kCopies = kGgElems * kBytes / 4096, kSize = kGgElems * kBytes;
    const uint8_t* base;
    int64_t stage;          // bytes from stage to stage
    uint32_t off[kCopies];
    int row, k;
    __device__ __forceinline__ static int swizzle(int row) { return COLS >= 128 ? row & 3 : COLS == 64 ? (row >> 1) & 1 : 0; }
    __device__ __forceinline__ void init(const uint8_t* b, int64_t stride, int cols, int contraction, int wave, int lane) {
        base = b;
        stage = kGgElems * stride;
        k = contraction;
        row = kRowsPer * wave + lane / kChunks;
        const int chunk = lane % kChunks ^ (swizzle(row) << 2);     // rows 4 kRowsPer apart have the same
#pragma unroll
        for (int q = 0; q < kCopies; ++q) off[q] = chunk * 8 < cols ? (uint32_t)((row + 4 * kRowsPer * q) * stride + chunk * 16) : kOutside;
    }
    __device__ __forceinline__ void issue(uint32_t lds, int s, int q, int wave) const {
        lds_copy16(buffer_desc(base + s * stage), __builtin_amdgcn_readfirstlane(lds + (4 * q + wave) * 1024),
                   s * kGgElems + row + 4 * kRowsPer * q < k ? off[q] : kOutside, 0u);
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

// ------------------------------------------------------------------ rows to workgroups
// An expert's rows as a workgroup needs them.
struct GgGroup {
    int e, first, rows, end;        // first row, rows with tokens, the end of its padding rows
    int tile, tiles;                // the block of the output among the expert's, its blocks of rows
};

__device__ __forceinline__ void gg_rows(const GgArgs& a, int e, int& first, int& rows, int& end) {
    // whatever the maps hold, rows stay inside [0, R) and an expert's inside its own
    const int R = (int)a.R, f = a.offsets[e], n = a.offsets[e + 1], c = a.counts[e];
    first = f < 0 ? 0 : f < R ? f : R;
    end = n < first ? first : n < R ? n : R;
    rows = c < 0 ? 0 : c < end - first ? c : end - first;
}

// XCD x (workgroups are dealt to the 8 round robin) gets a contiguous run of
// `total` blocks: which one this workgroup has, or -1.
__device__ __forceinline__ int xcd_run(int total) {
    const int x = blockIdx.x & 7, j = (int)(blockIdx.x >> 3), per = total >> 3, more = total & 7;
    return j < per + (x < more ? 1 : 0) ? x * per + (x < more ? x : more) + j : -1;
}

// The expert and block of this workgroup: experts in order, each with
// ceil(its rows / bm) x nt blocks. Every thread counts a few experts' blocks.
__device__ __forceinline__ bool gg_find(const GgArgs& a, int bm, int nt, GgGroup& out) {
    __shared__ int s_sum[4];
    __shared__ GgGroup s_out;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (a.E + 255) / 256, e0 = tid * per;
    int mine = 0;
    for (int i = 0; i < per; ++i) {
        if (e0 + i >= a.E) break;
        int first, rows, end;
        gg_rows(a, e0 + i, first, rows, end);
        mine += (end - first + bm - 1) / bm;
    }
    const int upto = wave_inclusive_scan(mine);
    if (lane == 63) s_sum[wave] = upto;
    if (tid == 0) s_out.e = -1;
    __syncthreads();
    int before = upto - mine;
    for (int w = 0; w < wave; ++w) before += s_sum[w];
    const int total = (s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3]) * nt;
    const int id = xcd_run(total);
    if (id < 0) return false;
    if (id >= before * nt && id < (before + mine) * nt) {
        for (int i = 0; i < per; ++i) {
            if (e0 + i >= a.E) break;
            GgGroup g;
            g.e = e0 + i;
            gg_rows(a, g.e, g.first, g.rows, g.end);
            g.tiles = (g.end - g.first + bm - 1) / bm;
            g.tile = id - before * nt;
            if (g.tile >= 0 && g.tile < g.tiles * nt) s_out = g;
            before += g.tiles;
        }
    }
    __syncthreads();
    out.e = __builtin_amdgcn_readfirstlane(s_out.e);
    if (out.e < 0) return false;
    out.first = __builtin_amdgcn_readfirstlane(s_out.first);
    out.rows = __builtin_amdgcn_readfirstlane(s_out.rows);
    out.end = __builtin_amdgcn_readfirstlane(s_out.end);
    out.tile = __builtin_amdgcn_readfirstlane(s_out.tile);
    out.tiles = __builtin_amdgcn_readfirstlane(s_out.tiles);
    return true;
}

// ------------------------------------------------------------------ output
template <int NW, bool F32>
constexpr int gg_row_bytes() { return 32 * NW * (F32 ? 4 : 2) + 16; }

// 32 rows of a wave's block: a lane holds 4 consecutive columns of one row at a
// time; the wave turns its NW tiles through its own part of the LDS and stores
// whole 16-byte pieces. Of `left` rows, those from `live` on are zeros.
template <int NW, bool F32, bool ADD>
__device__ __forceinline__ void gg_store(uint8_t* out, int64_t stride, bool vec, uint8_t* slab, const gg_f16v (&acc)[NW],
                                         int live, int left, int cols, int lane) {
    constexpr int kRow = gg_row_bytes<NW, F32>(), kEs = F32 ? 4 : 2, kPiece = 16 / kEs, kPieces = 32 * NW / kPiece;
    const int r = lane & 31, g = lane >> 5;
    wave_lds_sync();
#pragma unroll
    for (int n = 0; n < NW; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = 32 * n + 8 * q + 4 * g;
            floatx4 v = {acc[n][4 * q], acc[n][4 * q + 1], acc[n][4 * q + 2], acc[n][4 * q + 3]};
            if (r >= live) v = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (F32 || ADD) *reinterpret_cast<floatx4*>(slab + r * kRow + c * 4) = v;
            else *reinterpret_cast<uint2*>(slab + r * kRow + c * 2) = make_uint2(f32_to_bf16(v[0]) | (f32_to_bf16(v[1]) << 16),
                                                                                 f32_to_bf16(v[2]) | (f32_to_bf16(v[3]) << 16));
        }
    wave_lds_sync();
#pragma unroll 4
    for (int j = 0; j < 32 * kPieces / 64; ++j) {
        const int i = lane + 64 * j, row = i / kPieces, c = (i % kPieces) * kPiece;
        if (row >= left || c >= cols) continue;
        uint8_t* dst = out + row * stride + c * kEs;
        const uint8_t* src = slab + row * kRow + c * kEs;
        if (vec && c + kPiece <= cols) {
            *reinterpret_cast<u32x4*>(dst) = *reinterpret_cast<const u32x4*>(src);
        } else {
            for (int k = 0; k < kPiece && c + k < cols; ++k) {
                if constexpr (F32) reinterpret_cast<float*>(dst)[k] = reinterpret_cast<const float*>(src)[k];
                else reinterpret_cast<uint16_t*>(dst)[k] = reinterpret_cast<const uint16_t*>(src)[k];
            }
        }
    }
}

// The same for a sum onto what the output holds (bf16: added in fp32, rounded once).
template <int NW, bool F32>
__device__ __forceinline__ void gg_add(uint8_t* out, int64_t stride, uint8_t* slab, const gg_f16v (&acc)[NW], int left, int cols,
                                       int lane) {
    constexpr int kRow = gg_row_bytes<NW, true>();
    const int r = lane & 31, g = lane >> 5;
    wave_lds_sync();
#pragma unroll
    for (int n = 0; n < NW; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<floatx4*>(slab + r * kRow + (32 * n + 8 * q + 4 * g) * 4) =
                floatx4{acc[n][4 * q], acc[n][4 * q + 1], acc[n][4 * q + 2], acc[n][4 * q + 3]};
    wave_lds_sync();
#pragma unroll 8
    for (int j = 0; j < 32 * NW / 2; ++j) {
        const int i = lane + 64 * j, row = i / (32 * NW), c = i % (32 * NW);
        if (row >= left || c >= cols) continue;
        const float v = *reinterpret_cast<const float*>(slab + row * kRow + c * 4);
        if constexpr (F32) {
            float* dst = reinterpret_cast<float*>(out + row * stride) + c;
            *dst = __fadd_rn(*dst, v);
        } else {
            uint16_t* dst = reinterpret_cast<uint16_t*>(out + row * stride) + c;
            *dst = (uint16_t)f32_to_bf16(__fadd_rn(bf16_to_f32(*dst), v));
        }
    }
}

// ------------------------------------------------------------------ the kernel
// 4 waves, WM along the output's rows; a wave has MW x NW tiles of 32 x 32.
enum GgKind { kGgRows, kGgRowsT, kGgWeight };       // forward, input gradient, weight gradient

template <int KIND, int WM, int MW, int NW>
struct GgShape {
    static constexpr int kWN = 4 / WM, kBM = 32 * WM * MW, kBN = 32 * kWN * NW;
    using A = std::conditional_t<KIND == kGgWeight, Across<kBM>, Along<kBM>>;
    using B = std::conditional_t<KIND == kGgRows, Along<kBN>, Across<kBN>>;
    static constexpr int kAll = A::kCopies + B::kCopies, kStage = A::kSize + B::kSize;
    static constexpr int kPerCu = MW * NW >= 16 ? 1 : 2;
    static constexpr int kFit = (160 * 1024 / kPerCu - 256) / kStage, kRing = kFit < 6 ? kFit : 6;
    static_assert(kRing >= 2 && (kRing - 1) * kAll < 64, "ring of stages");
};

template <int KIND, int WM, int MW, int NW, bool F32, bool ADD>
__global__ void __launch_bounds__(256, (GgShape<KIND, WM, MW, NW>::kPerCu)) grouped_gemm_kernel(GgArgs a) {
    using S = GgShape<KIND, WM, MW, NW>;
    constexpr int kOutRow = gg_row_bytes<NW, F32 || ADD>(), kAll = S::kAll;
    constexpr int kLds = S::kRing * S::kStage > 4 * 32 * kOutRow ? S::kRing * S::kStage : 4 * 32 * kOutRow;
    __shared__ __align__(16) uint8_t lds[kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / S::kWN, wn = wave % S::kWN;

    GgGroup g;
    const int nt = (a.N + S::kBN - 1) / S::kBN;
    if constexpr (KIND == kGgWeight) {
        g.tiles = (a.M + S::kBM - 1) / S::kBM;
        const int id = xcd_run(a.E * g.tiles * nt);
        if (id < 0) return;
        g.e = id / (g.tiles * nt), g.tile = id - g.e * (g.tiles * nt);
        gg_rows(a, g.e, g.first, g.rows, g.end);
    } else {
        if (!gg_find(a, S::kBM, nt, g)) return;
    }
    // groups of 4 blocks of rows, column by column: what neighbours share stays in the XCD's L2
    const int gm0 = g.tile / (4 * nt) * 4, gh = g.tiles - gm0 < 4 ? g.tiles - gm0 : 4, in = g.tile - gm0 * nt;
    const int m0 = (gm0 + in % gh) * S::kBM, n0 = (in / gh) * S::kBN;

    typename S::A ca;
    typename S::B cb;
    int k, live, left;      // contraction; rows of the block that are computed, and that are written
    if constexpr (KIND == kGgWeight) {
        k = g.rows, live = left = a.M - m0;
        ca.init(a.a + g.first * a.a_stride + 2 * (int64_t)m0, a.a_stride, a.M - m0, k, wave, lane);
        cb.init(a.b + g.first * a.b_stride + 2 * (int64_t)n0, a.b_stride, a.N - n0, k, wave, lane);
    } else {
        live = g.rows - m0, left = g.end - g.first - m0;
        k = live > 0 ? a.K : 0;
        ca.init(a.a + (g.first + (int64_t)m0) * a.a_stride, a.a_stride, live, k, wave, lane);
        const uint8_t* b = a.b + g.e * a.b_group;
        if constexpr (KIND == kGgRows) cb.init(b + n0 * a.b_stride, a.b_stride, a.N - n0, k, wave, lane);
        else cb.init(b + 2 * (int64_t)n0, a.b_stride, a.N - n0, k, wave, lane);
    }
    if (ADD && k == 0) return;
    const int stages = (k + kGgElems - 1) / kGgElems;
    const uint32_t lds0 = lds_addr(lds);
    auto copy = [&](int s, int q0, int q1) {
        const uint32_t at = lds0 + (s % S::kRing) * S::kStage;
#pragma unroll
        for (int q = q0; q < q1; ++q) {
            if (q < S::A::kCopies) ca.issue(at, s, q, wave);
            else cb.issue(at + S::A::kSize, s, q - S::A::kCopies, wave);
        }
    };
    struct Operands {
        bf16x8 a[MW], b[NW];
    };
    auto read = [&](int s, int step, Operands& o) {
        const uint8_t* at = lds + (s % S::kRing) * S::kStage;
#pragma unroll
        for (int n = 0; n < NW; ++n) o.b[n] = S::B::read(at + S::A::kSize, wn * NW + n, step, lane);
#pragma unroll
        for (int m = 0; m < MW; ++m) o.a[m] = S::A::read(at, wm * MW + m, step, lane);
    };
    gg_f16v acc[MW][NW];
#pragma unroll
    for (int m = 0; m < MW; ++m)
#pragma unroll
        for (int n = 0; n < NW; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.0f;
    auto mfma = [&](const Operands& o, int m) {
#pragma unroll
        for (int n = 0; n < NW; ++n) acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(o.b[n], o.a[m], acc[m][n], 0, 0, 0);
    };
    auto mfmas = [&](const Operands& o) {
#pragma unroll
        for (int m = 0; m < MW; ++m) mfma(o, m);
        __builtin_amdgcn_sched_barrier(0);
    };

    // A ring of stages as in the MX product: one barrier a stage, in front of its
    // last step's MFMAs; every wave holds what it still needs of the stage by
    // then, and the copies of stage s + kRing go into its buffer behind it.
    if (stages > 0) {
#pragma unroll
        for (int s = 0; s < S::kRing; ++s) copy(s, 0, kAll);
        Operands o0, o1;
        __builtin_amdgcn_s_waitcnt(vmcnt_at_most((S::kRing - 1) * kAll));
        __syncthreads();
        read(0, 0, o0);
        for (int s = 0; s < stages; ++s) {
            read(s, 1, o1);
            mfmas(o0);
            read(s, 2, o0);
            mfmas(o1);
            read(s, 3, o1);
            mfmas(o0);
            __builtin_amdgcn_s_waitcnt(vmcnt_at_most((S::kRing - 2) * kAll) & lgkmcnt_zero());
            asm volatile("s_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            read(s + 1, 0, o0);
#pragma unroll
            for (int m = 0; m < MW; ++m) {
                copy(s + S::kRing, m * kAll / MW, (m + 1) * kAll / MW);
                mfma(o1, m);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // the copies of the stages behind the last still write (zeros) to the LDS
        __builtin_amdgcn_s_waitcnt(vmcnt_at_most(0) & lgkmcnt_zero());
        __syncthreads();
    }

    uint8_t* slab = lds + wave * 32 * kOutRow;
    const int c0 = n0 + 32 * NW * wn;
    const int es = F32 ? 4 : 2;
#pragma unroll
    for (int m = 0; m < MW; ++m) {
        const int r0 = 32 * (wm * MW + m);
        uint8_t* out = a.out + (KIND == kGgWeight ? g.e * a.out_group + (m0 + r0) * a.out_stride
                                                  : (g.first + (int64_t)m0 + r0) * a.out_stride) + (int64_t)c0 * es;
        if constexpr (ADD) gg_add<NW, F32>(out, a.out_stride, slab, acc[m], left - r0, a.N - c0, lane);
        else gg_store<NW, F32, false>(out, a.out_stride, a.out_vec, slab, acc[m], live - r0, left - r0, a.N - c0, lane);
    }
}

// ------------------------------------------------------------------ host side
template <int KIND, int WM, int MW, int NW>
int launch_grouped(const GgArgs& a, bool f32, bool add, hipStream_t s, const char* name) {
    using S = GgShape<KIND, WM, MW, NW>;
    const int64_t nt = (a.N + S::kBN - 1) / S::kBN;
    int64_t tiles;
    if (KIND == kGgWeight) tiles = (int64_t)a.E * ((a.M + S::kBM - 1) / S::kBM) * nt;
    else tiles = (a.R / S::kBM + (a.R < a.E ? a.R : a.E)) * nt;     // whole blocks, and each expert's last
    if (!launch_fits(tiles, 256)) return fail(MOE_EUNSUPPORTED, "%s: too many output tiles", name);
    const dim3 g((unsigned)tiles), b(256);
    if constexpr (KIND == kGgWeight) {
        if (add) {
            if (f32) hipLaunchKernelGGL((grouped_gemm_kernel<KIND, WM, MW, NW, true, true>), g, b, 0, s, a);
            else hipLaunchKernelGGL((grouped_gemm_kernel<KIND, WM, MW, NW, false, true>), g, b, 0, s, a);
            return check_launch(name);
        }
    }
    if (f32) hipLaunchKernelGGL((grouped_gemm_kernel<KIND, WM, MW, NW, true, false>), g, b, 0, s, a);
    else hipLaunchKernelGGL((grouped_gemm_kernel<KIND, WM, MW, NW, false, false>), g, b, 0, s, a);
    return check_launch(name);
}

// Sizes of the three calls.
static int gg_sizes(int64_t rows_max, int E, int N, int D, int dtype, const char* name) {
    if (rows_max < 0 || rows_max > 0x7FFFFFFF || E < 1 || E > MOE_MAX_EXPERTS || N < 0 || D < 0)
        return fail(MOE_EINVAL, "%s: rows_max=%lld E=%d N=%d D=%d out of range", name, (long long)rows_max, E, N, D);
    if (dtype != MOE_BF16 && dtype != MOE_F32)
        return fail(MOE_EINVAL, "%s: dtype %d is neither MOE_BF16 nor MOE_F32", name, dtype);
    if (N % 8 || D % 8 || N > MOE_MAX_GROUPED || D > MOE_MAX_GROUPED)
        return fail(MOE_EUNSUPPORTED, "%s: N=%d and D=%d must be multiples of 8 up to %d", name, N, D, MOE_MAX_GROUPED);
    return MOE_OK;
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
    if (gg_bad_stride(x_row_stride, in_cols) || out_row_stride < out_cols)
        return fail(MOE_EINVAL, "%s: row strides must be >= the rows (the input's a multiple of 8, at most %d)", name, 1 << 21);
    GgArgs a{};
    a.a = (const uint8_t*)x; a.a_stride = 2 * x_row_stride;
    a.b = (const uint8_t*)w; a.b_stride = 2 * (int64_t)D; a.b_group = 2 * (int64_t)N * D;
    a.offsets = offsets; a.counts = counts; a.E = E; a.R = rows_max; a.N = out_cols; a.K = in_cols;
    const bool f32 = out_dtype == MOE_F32;
    a.out = (uint8_t*)out; a.out_stride = out_row_stride * (f32 ? 4 : 2); a.out_vec = a.out_stride % 16 == 0;
    hipStream_t s = (hipStream_t)stream;
    if (rows_max >= 128 * (int64_t)E)
        return input_grad ? launch_grouped<kGgRowsT, 2, 4, 4>(a, f32, false, s, name) : launch_grouped<kGgRows, 2, 4, 4>(a, f32, false, s, name);
    return input_grad ? launch_grouped<kGgRowsT, 1, 1, 1>(a, f32, false, s, name) : launch_grouped<kGgRows, 1, 1, 1>(a, f32, false, s, name);
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
    if ((int64_t)E * ((N + 127) / 128) * ((D + 127) / 128) >= 256)
        return launch_grouped<kGgWeight, 2, 4, 4>(a, f32, accumulate != 0, (hipStream_t)stream, name);
    return launch_grouped<kGgWeight, 2, 1, 1>(a, f32, accumulate != 0, (hipStream_t)stream, name);
}
