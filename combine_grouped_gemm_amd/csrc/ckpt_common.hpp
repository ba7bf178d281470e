// The 8-bit checkpoint format: int8 codes and a power-of-two scale for each
// block of 128 columns of a row.
//
// s = the smallest 2^e, -126 <= e <= 121, with amax <= 127 s (1 for a block of
// zeros); code = v / s to the nearest integer, ties to even, within +-127.
// v / s is exact (a power of two), so one fma onto 1.5 * 2^23 rounds it once
// and leaves the code in its low byte.  Only a block whose amax lies above 127 *
// 2^121 can reach 128 and is held at 127.  code * s has 7 significant bits and
// an exponent that bf16 has: every product that takes a checkpoint takes it
// exactly.  A block with a NaN or an infinity gets scale NaN and codes 0, so
// what is computed from it is NaN.
#pragma once

#include "device_common.hpp"

namespace moeep {

constexpr int kCkptBlock = 128;

// Scale of a block whose largest magnitude has the bits `amax` (sign cleared).
// 127 = 1.984375 * 2^6: amax = m * 2^E needs 2^(E - 6) if its fraction is at
// most that of 127, else 2^(E - 5).
__device__ __forceinline__ float ckpt_scale(uint32_t amax) {
    if (amax == 0u) return 1.0f;
    if (amax >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    int e = (int)(amax >> 23) - 6 + ((amax & 0x7fffffu) > 0x7e0000u ? 1 : 0);     // biased
    e = e < 1 ? 1 : (e > 248 ? 248 : e);
    return __uint_as_float((uint32_t)e << 23);
}

// 1 / s for a scale of ckpt_scale: 2^-e, also a normal number (NaN stays NaN)
__device__ __forceinline__ float ckpt_recip(float s) {
    const uint32_t u = __float_as_uint(s);
    return u >= 0x7f800000u ? s : __uint_as_float(0x7f000000u - u);
}

// The code of v in the low byte; s NaN: 0.
__device__ __forceinline__ uint32_t ckpt_code(float v, float rs) {
    constexpr float kMagic = 12582912.0f;                                         // 1.5 * 2^23
    const float t = fminf(fmaxf(fmaf(v, rs, kMagic), kMagic - 127.0f), kMagic + 127.0f);
    return __float_as_uint(t);
}

// low bytes of four words, first in bits 7:0
__device__ __forceinline__ uint32_t pack_low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_amdgcn_perm(b, a, 0x0c0c0400u) | __builtin_amdgcn_perm(d, c, 0x04000c0cu);
}

// the codes of four neighbouring columns under scale s
__device__ __forceinline__ uint32_t ckpt_codes4(const floatx4& v, float s) {
    const float rs = ckpt_recip(s);
    const uint32_t q = pack_low_bytes(ckpt_code(v[0], rs), ckpt_code(v[1], rs), ckpt_code(v[2], rs), ckpt_code(v[3], rs));
    return s == s ? q : 0u;
}

// the value of byte k of w as a signed code
template <int k>
__device__ __forceinline__ float code_value(uint32_t w) {
    return (float)((int)(w << (24 - 8 * k)) >> 24);
}

// Maximum over the 16 lanes of a DPP row (as row16_max, for bit patterns).
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
    auto most = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    v = most(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
    v = most(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
    v = most(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));
    v = most(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));
    return v;
}

// By groups of 16 lanes: even groups keep a and get the next group's a as b, odd groups get the
// group before's b as a and keep b.
__device__ __forceinline__ void exchange_groups_u32(uint32_t& a, uint32_t& b) {
#if defined(__HIP_DEVICE_COMPILE__)
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
#endif
}

// Maxima over the four lanes l, l + 16, l + 32, l + 48: of a in lanes 0..31, of b in 32..63.
__device__ __forceinline__ uint32_t lane_groups_max(uint32_t a, uint32_t b) {
#if defined(__HIP_DEVICE_COMPILE__)
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    const uint32_t m = r[0] > r[1] ? r[0] : r[1];
    const auto q = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    return q[0] > q[1] ? q[0] : q[1];
#else
    return 0u;
#endif
}

}  // namespace moeep
