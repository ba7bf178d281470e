// Grouped SwiGLU expert FFN with int8 operands: one fp32 scale per token (row)
// and one per output channel (weight row), int32 accumulation on MFMA.
//
//   gate/up:  g[r,n] = sx[r] swg[n] sum_k x[r,k] wg[n,k],  u likewise,
//             h = silu(g) * u, rounded once to bf16
//   down:     y[r,n] = sh[r] swd[n] sum_k h[r,k] wd[n,k], bf16 or fp32
//
// The int32 sums are exact (|sum| <= 2^14 K < 2^31, the host bounds K), so the
// only roundings are the sum's conversion to fp32, the two scalings and the
// one to the output type, and results do not depend on the tile shape.  Scales
// factor out of the contraction, so the k loop holds nothing but loads and
// v_mfma_i32_16x16x64_i8: lane l feeds row (l % 16) with the 16 bytes of
// k-chunk (l / 16) for both operands and receives rows 4*(l/16)+i, column
// l % 16 of the 16x16 result, the bf16 instruction's layout byte for byte.
//
// h leaves gate/up as bf16, not int8: its scale is the largest magnitude of a
// whole row, which many tiles write; moe_quant_rows makes the int8 rows.
#include "gemm_wide_i8.hpp"

namespace moeep {
namespace {

template <int BM, int BN, int S, bool GATED, bool OUT_F32, bool NT_W>
hipError_t launch_wide(const FfnArgs& a, hipStream_t stream) {
    static int per_cu = 0;
    return launch_persistent(widei8::grouped_gemm_i8_wide_kernel<BM, BN, S, GATED, OUT_F32, NT_W>, 512, a, stream,
                             &per_cu);
}

// The weights' cache policy.  Read with the non-temporal hint they leave L2 at
// once: faster where each line is read by one tile (2 rows per expert of the
// DeepSeek-shaped layer, gate/up 944 us against 1062; EP share, 115 rows, 179
// against 188; 64-row tiles on 10-60 rows 1-3%).  Rows that are no whole number of
// 128-byte lines need each line in two k-steps (H = I = 2880, 128 rows: 284 us
// without the hint, 337 with it), and experts with more rows than a tile have their
// weights read again by the next tile (256 rows 2188 us without, 2201 with; 64-row
// tiles on 100 rows 6-14% faster without, on 600 rows 11-14%).
template <int BM, int BN, int S>
hipError_t launch_out(const FfnArgs& a, bool gated, hipStream_t stream) {
    const bool nt = a.ldw % 128 == 0 && a.rows_hint < BM * 3 / 4;
    if (gated) return nt ? launch_wide<BM, BN, S, true, false, true>(a, stream) : launch_wide<BM, BN, S, true, false, false>(a, stream);
    if (a.out_f32) return nt ? launch_wide<BM, BN, S, false, true, true>(a, stream) : launch_wide<BM, BN, S, false, true, false>(a, stream);
    return nt ? launch_wide<BM, BN, S, false, false, true>(a, stream) : launch_wide<BM, BN, S, false, false, false>(a, stream);
}

}  // namespace

// Tile shape.  Few rows per expert: 64 x 128 tiles in three stages, two workgroups
// per CU (4 rows, all 256 experts with some: gate/up 1061 us against 1088 with 256 x
// 256, down 569 against 599; 16 rows at H = I = 2880: gate/up 399 against 409).
// Many: 256 x 256 (64 rows: 1337 us against 1648; 256: 2147 against 3646).  They meet
// at about 32 (1197 against 1201 at H = 7168, down 735 against 721; 432 against 437 at
// 2880).  However many rows there are, large tiles that leave CUs without one lose to
// small ones that all run at once: 8 experts of 180 rows, 768 columns of 7168, 24
// large tiles 72 us, 144 small 34; 250 rows, 2048 columns, 64 large 89, 512 small 58;
// where the large ones number half the CUs they are even (100 rows, gate and up of
// 2048 columns, 128 large 64 us, 512 small 67).  Past one round of small tiles: 16
// such experts 81 against 119.
// Two stages instead of three under the small tile gain 0.1-0.2 us of 5 where
// fewer than some 200 tiles take one or two steps each, and lose 5-25% where more do
// (256 experts of 512 columns, K = 144: 12.7 us, 15.2 with two).
hipError_t launch_ffn_i8(const FfnArgs& a, bool gated, hipStream_t stream) {
    constexpr int BM = 64, BN = 128;
    const int cols = gated ? BN / 2 : BN;
    const long long row_tiles = ((long long)a.rows_hint + BM - 1) / BM;
    const long long small = a.E_loc * row_tiles * ((a.N + cols - 1) / cols);
    if (a.rows_hint >= 32 && small > 2 * device_cu_count()) return launch_out<256, 256, 2>(a, gated, stream);
    return launch_out<BM, BN, 3>(a, gated, stream);
}

}  // namespace moeep
