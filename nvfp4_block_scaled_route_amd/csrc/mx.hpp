// OCP microscaling (MX) blocks: 32 consecutive elements of a row under one
// e8m0 scale byte b, the value 2^(b - 127) (255: NaN).
#pragma once
#include "common.hpp"

namespace moe {

constexpr int kMxBlock = 32;

inline bool mx_fmt_ok(int fmt) { return fmt == MOE_MX_E2M1 || fmt == MOE_MX_E4M3; }
// bytes that n elements take (n a multiple of 32)
__host__ __device__ __forceinline__ int64_t mx_bytes(int64_t n, int fmt) {
    return fmt == MOE_MX_E2M1 ? n >> 1 : n;
}

// The exponent of a format's largest binade: 4 <= 6 < 8, 256 <= 448 < 512.
template <int FMT>
__device__ __forceinline__ constexpr int mx_emax() { return FMT == MOE_MX_E2M1 ? 2 : 8; }

// The maximum over the 4 lanes of a quad, in all four.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    const uint32_t a = (uint32_t)dpp_i<kDppQuadXor1>((int)v);
    v = v > a ? v : a;
    const uint32_t b = (uint32_t)dpp_i<kDppQuadXor2>((int)v);
    return v > b ? v : b;
}

// The scale byte of a block from the bits of its largest magnitude: the
// magnitude's exponent less the format's (a block of zeros, or of magnitudes
// below the smallest scale's reach: byte 0), 255 if it is infinite or NaN.
// Magnitudes compare as their bits (a NaN is above infinity), so one maximum
// over the bits finds both the block's amax and whether it is finite.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 23);
    if (e == 255) return 255u;
    const int b = e - mx_emax<FMT>();
    return (uint32_t)(b > 0 ? b : 0);
}

// 2^(127 - byte), what the elements are multiplied with: a normal fp32 number
// for every byte below 254 (finite amax gives at most 252), and 0 for 255, so
// that a NaN block's codes are cleared after the product.
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 8 fp32 values of a block -> their codes (8 bytes, or 4 in .x). The scaled
// magnitudes are below 2 * 2^emax, so saturating is the only clamp. The
// hardware's pack conversions round to nearest even and keep the sign of zero;
// the one to e2m1 saturates by itself, the one to e4m3 does not.
template <int FMT>
__device__ __forceinline__ uint2 mx_codes8(const float (&v)[8], uint32_t byte) {
    if (byte == 255u) return make_uint2(0u, 0u);
    const float m = mx_inv_scale(byte);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fmul_rn(v[i], m);
    if constexpr (FMT == MOE_MX_E2M1) {
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[0], q[1], 1.0f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[2], q[3], 1.0f, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[4], q[5], 1.0f, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[6], q[7], 1.0f, 3);
        return make_uint2(w, 0u);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf(q[i], -448.0f), 448.0f);
        int lo = 0, hi = 0;
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
        return make_uint2((uint32_t)lo, (uint32_t)hi);
    }
}

// 8 bf16 values (16 bytes) -> fp32.
__device__ __forceinline__ void unpack8(const uint4& p, float (&v)[8]) {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t amax8_bits(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        m = m > b ? m : b;
    }
    return m;
}

// Lane's 8 values (a quad holds one block, in order) -> codes and scale byte at
// octet `oct` from codes and sf on.
template <int FMT>
__device__ __forceinline__ void mx_store8(const float (&v)[8], int64_t oct, uint8_t* codes, uint8_t* sf) {
    const uint32_t byte = mx_scale_byte<FMT>(quad_max(amax8_bits(v)));
    const uint2 c = mx_codes8<FMT>(v, byte);
    if constexpr (FMT == MOE_MX_E2M1) *reinterpret_cast<uint32_t*>(codes + oct * 4) = c.x;
    else *reinterpret_cast<uint2*>(codes + oct * 8) = c;
    if ((oct & 3) == 0) sf[oct >> 2] = (uint8_t)byte;
}

}  // namespace moe
