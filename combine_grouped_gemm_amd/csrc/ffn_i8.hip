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
// once: 5% faster where each line is read by one tile (T = 64 decode 857 against
// 887 us, EP share 209 against 219).  Rows that are no whole number of 128-byte
// lines need each line in two k-steps (H = I = 2880: 300 us without the hint,
// 342 with it), and experts with more rows than a tile have their weights read
// again by the next tile (256 rows prefill 2085 us without, 2133 with it; 64-row
// tiles on 100 rows 3-8% faster without, on 600 rows 9-18%; on 40 rows, one tile,
// 5-9% slower).
template <int BM, int BN, int S>
hipError_t launch_out(const FfnArgs& a, bool gated, hipStream_t stream) {
    const bool nt = a.ldw % 128 == 0 && a.rows_hint < BM * 3 / 4;
    if (gated) return nt ? launch_wide<BM, BN, S, true, false, true>(a, stream) : launch_wide<BM, BN, S, true, false, false>(a, stream);
    if (a.out_f32) return nt ? launch_wide<BM, BN, S, false, true, true>(a, stream) : launch_wide<BM, BN, S, false, true, false>(a, stream);
    return nt ? launch_wide<BM, BN, S, false, false, true>(a, stream) : launch_wide<BM, BN, S, false, false, false>(a, stream);
}

}  // namespace

// Tile shape.  Few rows per expert: 64 x 128 tiles, two workgroups per CU (T = 128
// decode gate/up 1003 us against 1022 us with 256 x 256, down 524 against 538; 16
// rows per expert at H = I = 2880: 447 against 475).  Many: 256 x 256 (64 rows per
// expert: 1285 us against 1663; 256: 2120 against 5180).  They meet at about 32
// (1194 against 1257 at H = 7168, 482 against 487 at 2880); 128 x 128 tiles were
// never better than both by more than 1.5%.  However many rows there are, large
// tiles that leave CUs without one lose to small ones that all run at once: 8
// experts of 180 rows, 768 columns of 7168, 24 large tiles 64 us, 144 small 33;
// 250 rows, 2048 columns, 64 large 79, 512 small 57; 100 rows, gate and up of 2048
// columns, 128 large 72.5, 512 small 68.  Past one round of small tiles: 16 such
// experts 84 against 129.
hipError_t launch_ffn_i8(const FfnArgs& a, bool gated, hipStream_t stream) {
    constexpr int BM = 64, BN = 128;
    const int cols = gated ? BN / 2 : BN;
    const long long row_tiles = ((long long)a.rows_hint + BM - 1) / BM;
    const long long small = a.E_loc * row_tiles * ((a.N + cols - 1) / cols);
    if (a.rows_hint >= 32 && small > 2 * device_cu_count()) return launch_out<256, 256, 2>(a, gated, stream);
    // two steps have nothing for a third stage (31 experts, K = 144, 14.7 us against 16.6)
    return a.Kdim > 2 * widei8::BK ? launch_out<BM, BN, 3>(a, gated, stream) : launch_out<BM, BN, 2>(a, gated, stream);
}

}  // namespace moeep
