// Operands of the gradient products whose contraction runs over the rows of a
// row-major matrix: weights (out, in) of an input gradient, both operands of a
// weight gradient.  Their k-step sits in LDS as it is in memory, [k][columns], and a
// lane of a matrix instruction needs consecutive k of one column: gfx950's transposing
// read (ds_read_b64_tr_b16) gives it that.  Each group of 16 lanes reads four rows of
// 16 columns, 8 bytes a lane (lane i: row i / 4, columns 4 (i % 4) ...), and lane i
// receives the four rows' values of column i.
//
// A v_mfma_f32_16x16x32_bf16 lane l feeds column l % 16 with k = 8 (l / 16) .. + 7, so
// a fragment is two such reads, rows 8 g + 0..3 and 8 g + 4..7 of the 32-row half (g = l
// / 16).  A row's 32-byte column pairs are permuted by XOR with (k & 3) | ((k >> 3) <<
// 2), as many bits as the row has pairs: the 16 rows a read touches then lie in distinct
// banks, and the permutation does not change between a fragment's two reads or between
// the two halves of a 64-row step, so that they differ by constant offsets.
#pragma once

#include "gemm_wide.hpp"

namespace moeep {
namespace cols {

using namespace wide;

// XOR of a row's 16-byte chunk index, for rows of TW columns (TW / 8 chunks)
template <int TW>
__device__ __forceinline__ int swz_row(int k) {
    constexpr int kBits = TW == 256 ? 3 : 1;
    static_assert(TW == 256 || TW == 128, "row width");
    return 2 * ((k & 3) | (((k >> 3) & kBits) << 2));
}

// byte offset in a [64][TW] stage of what lane l reads for the fragment of columns
// [c0, c0 + 16), first half, rows 8 g + 0..3; the second half lies 32 rows further, rows
// 8 g + 4..7 four rows
template <int TW>
__device__ __forceinline__ uint32_t frag_offset(int lane, int c0) {
    const int i = lane & 15, k = (lane >> 4) * 8 + (i >> 2);
    return (uint32_t)(k * TW * 2 + (((c0 >> 3) + ((i & 3) >> 1)) ^ swz_row<TW>(k)) * 16 + (i & 1) * 8);
}

// the first k of a fragment's two reads in its low half
__device__ __forceinline__ bf16x8 join_frag(uint2 lo, uint2 hi) {
    return __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
}

typedef short shortx4 __attribute__((ext_vector_type(4)));

// one fragment by the builtin (the compiler places the wait)
template <int TW>
__device__ __forceinline__ bf16x8 read_frag(const char* stage, uint32_t off, int half) {
#if defined(__HIP_DEVICE_COMPILE__)
    typedef __attribute__((address_space(3))) shortx4* lds4;
    const char* p = stage + off + half * 32 * TW * 2;
    const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)p);
    const shortx4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 4 * TW * 2));
    return join_frag(__builtin_bit_cast(uint2, lo), __builtin_bit_cast(uint2, hi));
#else
    return bf16x8{};
#endif
}

// Fragments of one 32-row half of a [64][TW] stage, read and waited for in one block (as
// lds_read16x4): ad holds the LDS addresses of their first reads in the first half.
template <int TW, int HALF>
__device__ __forceinline__ void read_frags(bf16x8 (&f)[4], const uint32_t (&ad)[4]) {
    uint2 t[8];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8 offset:%12\n\t"
        "ds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
        "ds_read_b64_tr_b16 %2, %9 offset:%12\n\t"
        "ds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
        "ds_read_b64_tr_b16 %4, %10 offset:%12\n\t"
        "ds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
        "ds_read_b64_tr_b16 %6, %11 offset:%12\n\t"
        "ds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(t[0]), "=&v"(t[1]), "=&v"(t[2]), "=&v"(t[3]), "=&v"(t[4]), "=&v"(t[5]), "=&v"(t[6]), "=&v"(t[7])
        : "v"(ad[0]), "v"(ad[1]), "v"(ad[2]), "v"(ad[3]), "n"(HALF * 32 * TW * 2), "n"((HALF * 32 + 4) * TW * 2)
        : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = join_frag(t[2 * i], t[2 * i + 1]);
}
template <int TW, int HALF>
__device__ __forceinline__ void read_frags(bf16x8 (&f)[2], const uint32_t (&ad)[2]) {
    uint2 t[4];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4 offset:%6\n\t"
        "ds_read_b64_tr_b16 %1, %4 offset:%7\n\t"
        "ds_read_b64_tr_b16 %2, %5 offset:%6\n\t"
        "ds_read_b64_tr_b16 %3, %5 offset:%7\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(t[0]), "=&v"(t[1]), "=&v"(t[2]), "=&v"(t[3])
        : "v"(ad[0]), "v"(ad[1]), "n"(HALF * 32 * TW * 2), "n"((HALF * 32 + 4) * TW * 2)
        : "memory");
#pragma unroll
    for (int i = 0; i < 2; ++i) f[i] = join_frag(t[2 * i], t[2 * i + 1]);
}

// Of two fragments' results (lane n of 16 has row n of each): a becomes rows 0..7 of both, the
// second's in lanes 8..15, b rows 8..15, the first's in lanes 0..7.
__device__ __forceinline__ void exchange_rows(float& a, float& b) {
    const int x = __float_as_int(a), y = __float_as_int(b);
    constexpr int kRor8 = 0x128;
    a = __int_as_float(__builtin_amdgcn_update_dpp(x, y, kRor8, 0xf, 0xc, false));
    b = __int_as_float(__builtin_amdgcn_update_dpp(y, x, kRor8, 0xf, 0x3, false));
}
__device__ __forceinline__ void exchange_groups(float& a, float& b) {
    uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    exchange_groups_u32(x, y);
    a = __uint_as_float(x);
    b = __uint_as_float(y);
}

// 16 rows by 64 columns of a wave (four fragments, the columns as the matrix instructions' row
// operand) as bf16 in two 16-byte units a lane: unit h is row 8 h + l % 8, columns unit_col(l) ..
// + 7, so that 8 lanes hold a row's 128 bytes.
__device__ __forceinline__ int unit_col(int lane) {
    return ((lane >> 3) & 1) * 16 + ((lane >> 4) & 1) * 32 + (lane >> 5) * 8;
}
__device__ __forceinline__ void units_of(const floatx4 (&acc)[4], uint4 (&unit)[2]) {
    float t[4][4];
#pragma unroll
    for (int f = 0; f < 4; f += 2)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            t[f][e] = acc[f][e];
            t[f + 1][e] = acc[f + 1][e];
            exchange_rows(t[f][e], t[f + 1][e]);
        }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int e = 0; e < 4; ++e) exchange_groups(t[h][e], t[h + 2][e]);
        unit[h] = make_uint4(pack_bf16x2(t[h][0], t[h][1]), pack_bf16x2(t[h][2], t[h][3]),
                             pack_bf16x2(t[h + 2][0], t[h + 2][1]), pack_bf16x2(t[h + 2][2], t[h + 2][3]));
    }
}

// quotient of a slot by the slots of a token, exact for slots below 2^31: the host's
// multiplier and shift (divisor_of in launch.hpp)
__device__ __forceinline__ int token_of(int slot, const Divisor& d) {
    return d.shift < 0 ? slot : (int)(__umulhi((uint32_t)slot, d.mul) >> d.shift);
}

}  // namespace cols
}  // namespace moeep
