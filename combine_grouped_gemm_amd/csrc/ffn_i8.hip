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
#include "grouped_tiles.hpp"

namespace moeep {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));

// Register-staged tile: K loop in steps of 128 bytes per row, global 16-byte
// loads one step ahead (non-temporal for the weights), LDS chunks
// XOR-swizzled by (row & 7).
template <int BM, int BN, int WMW, int WNW, bool GATED, bool OUT_F32>
__global__ __launch_bounds__(64 * WMW * WNW) void grouped_gemm_i8_kernel(FfnArgs p) {
    constexpr int NT = 64 * WMW * WNW;
    constexpr int FM = BM / 16 / WMW;          // m-fragments per wave
    constexpr int WN = BN / WNW;               // B-tile rows per wave
    constexpr int FN = WN / 16;                // n-fragments per wave
    constexpr int BNO = GATED ? BN / 2 : BN;   // output columns per tile
    static_assert(FM >= 1 && FN >= 1 && (!GATED || FN % 2 == 0), "tile shape");
    constexpr int A_IT = (BM * 8 + NT - 1) / NT;
    constexpr int B_IT = (BN * 8 + NT - 1) / NT;

    __shared__ uint4 sA[BM * 8];
    __shared__ uint4 sB[BN * 8];
    __shared__ int s_pre[kMaxExperts + 1];
    __shared__ int s_tmp[NT / kWave];

    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int wm = wave / WNW, wn = wave % WNW;
    const int Kdim = p.Kdim, N = p.N, ldw = p.ldw;

    build_tile_prefix<NT, BM>(p, s_pre, s_tmp);
    const int n_tiles_n = (N + BNO - 1) / BNO;
    const int total = n_tiles_n * s_pre[p.E_loc];
    const int G = gridDim.x;
    const int v = xcd_block_order();

    const uint8_t* __restrict__ A = static_cast<const uint8_t*>(p.a);
    const uint8_t* __restrict__ W0 = static_cast<const uint8_t*>(p.w0);
    const uint8_t* __restrict__ W1 = static_cast<const uint8_t*>(p.w1);

    for (int rnd = 0;; ++rnd) {
        const int tau = round_tile(rnd, v, blockIdx.x, G, total);
        if (tau < 0) break;
        const TileCoord tc = decode_tile<BM>(tau, n_tiles_n, s_pre, p);
        const int j = tc.j, row0 = tc.row0, nvalid = tc.nvalid;
        const int col0 = tc.nt * BNO;
        const uint8_t* wg = W0 + (size_t)j * N * ldw;
        const uint8_t* wu = GATED ? W1 + (size_t)j * N * ldw : nullptr;

        uint4 ra[A_IT], rb[B_IT];
#pragma unroll
        for (int i = 0; i < A_IT; ++i) ra[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < B_IT; ++i) rb[i] = make_uint4(0, 0, 0, 0);
        auto load_step = [&](int k0) {
#pragma unroll
            for (int i = 0; i < A_IT; ++i) {
                const int q = tid + i * NT;
                const int r = q >> 3, c = q & 7;
                // chunks past K (a partial last step) are zero
                if (q < BM * 8 && r < nvalid)
                    ra[i] = k0 + c * 16 < Kdim
                                ? *reinterpret_cast<const uint4*>(A + (size_t)(row0 + r) * Kdim + k0 + c * 16)
                                : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < B_IT; ++i) {
                const int q = tid + i * NT;
                const int r = q >> 3, c = q & 7;
                if (q < BN * 8) {
                    const bool up = GATED && r >= BN / 2;
                    const int col = col0 + (up ? r - BN / 2 : r);
                    const uint8_t* src = up ? wu : wg;
                    if (col < N)
                        rb[i] = k0 + c * 16 < Kdim ? load_stream16(src + (size_t)col * ldw + k0 + c * 16)
                                                   : make_uint4(0, 0, 0, 0);
                }
            }
        };
        auto store_step = [&]() {
#pragma unroll
            for (int i = 0; i < A_IT; ++i) {
                const int q = tid + i * NT;
                const int r = q >> 3, c = q & 7;
                if (q < BM * 8 && r < nvalid) sA[r * 8 + (c ^ (r & 7))] = ra[i];
            }
#pragma unroll
            for (int i = 0; i < B_IT; ++i) {
                const int q = tid + i * NT;
                const int r = q >> 3, c = q & 7;
                if (q < BN * 8) sB[r * 8 + (c ^ (r & 7))] = rb[i];
            }
        };

        intx4 acc[FM][FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int f = 0; f < FN; ++f) acc[i][f] = intx4{0, 0, 0, 0};

        auto brow = [&](int f) {       // B-tile row of this lane for n-fragment f
            if (GATED) {
                const int half = f < FN / 2 ? 0 : BN / 2;
                const int ff = f < FN / 2 ? f : f - FN / 2;
                return half + wn * (WN / 2) + ff * 16 + (lane & 15);
            }
            return wn * WN + f * 16 + (lane & 15);
        };
        auto fcol = [&](int f) {       // output column of fragment f's first lane column
            if (GATED) {
                const int ff = f < FN / 2 ? f : f - FN / 2;
                return col0 + wn * (WN / 2) + ff * 16;
            }
            return col0 + wn * WN + f * 16;
        };

        load_step(0);
        for (int k0 = 0; k0 < Kdim; k0 += 128) {
            __syncthreads();
            store_step();
            __syncthreads();
            if (k0 + 128 < Kdim) load_step(k0 + 128);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const int chunk = kk * 4 + (lane >> 4);
                intx4 bfr[FN];
#pragma unroll
                for (int f = 0; f < FN; ++f) {
                    const int r = brow(f);
                    bfr[f] = __builtin_bit_cast(intx4, sB[r * 8 + (chunk ^ (r & 7))]);
                }
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const int mrow = (wm + WMW * i) * 16;
                    if (mrow < nvalid) {
                        const int r = mrow + (lane & 15);
                        const intx4 afr = __builtin_bit_cast(intx4, sA[r * 8 + (chunk ^ (r & 7))]);
#pragma unroll
                        for (int f = 0; f < FN; ++f)
                            if (fcol(f) < N)
                                acc[i][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(afr, bfr[f], acc[i][f], 0, 0, 0);
                    }
                }
            }
        }

        constexpr int FO = GATED ? FN / 2 : FN;
#pragma unroll
        for (int f = 0; f < FO; ++f) {
            const int col = fcol(f) + (lane & 15);
            if (col >= N) continue;
            const float sg = p.w0_scales[(size_t)j * N + col];
            const float su = GATED ? p.w1_scales[(size_t)j * N + col] : 0.0f;
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int mrow = (wm + WMW * i) * 16;
                if (mrow >= nvalid) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = mrow + (lane >> 4) * 4 + e;
                    if (r >= nvalid) continue;
                    const float sa = p.a_scales[row0 + r];
                    float val = (float)acc[i][f][e] * sa * sg;
                    if (GATED) val = silu(val) * ((float)acc[i][f + FN / 2][e] * sa * su);
                    const size_t at = (size_t)(row0 + r) * N + col;
                    if (OUT_F32) static_cast<float*>(p.out)[at] = val;
                    else static_cast<uint16_t*>(p.out)[at] = (uint16_t)f32_to_bf16_bits(val);
                }
            }
        }
    }
}

template <int BM, int BN, int WMW, int WNW, bool GATED, bool OUT_F32>
hipError_t launch_cfg(const FfnArgs& a, hipStream_t stream) {
    static int per_cu = 0;
    return launch_persistent(grouped_gemm_i8_kernel<BM, BN, WMW, WNW, GATED, OUT_F32>, 64 * WMW * WNW, a, stream,
                             &per_cu);
}

template <int BM, bool GATED, bool OUT_F32>
hipError_t launch_wide(const FfnArgs& a, hipStream_t stream) {
    static int per_cu = 0;
    return launch_persistent(widei8::grouped_gemm_i8_wide_kernel<BM, GATED, OUT_F32>, 512, a, stream, &per_cu);
}

template <int BM>
hipError_t launch_wide_any(const FfnArgs& a, bool gated, hipStream_t stream) {
    if (gated) return launch_wide<BM, true, false>(a, stream);
    return a.out_f32 ? launch_wide<BM, false, true>(a, stream) : launch_wide<BM, false, false>(a, stream);
}

}  // namespace

hipError_t launch_ffn_i8(const FfnArgs& a, bool gated, hipStream_t stream) {
    // the wide kernels address one expert's weight matrix with 32-bit offsets
    // and keep every resource extent (plus the k-step offset) below 2^31, so
    // that an out-of-range lane offset exists
    const bool wide_ok = (unsigned long long)a.N * a.ldw < (1ull << 31) &&
                         (unsigned long long)320 * (a.Kdim + 128) < (1ull << 31);
    if (wide_ok && a.rows_hint >= 192) return launch_wide_any<320>(a, gated, stream);
    if (wide_ok && a.rows_hint >= 64) return launch_wide_any<256>(a, gated, stream);
    if (gated) return launch_cfg<128, 128, 2, 2, true, false>(a, stream);
    return a.out_f32 ? launch_cfg<128, 128, 2, 2, false, true>(a, stream)
                     : launch_cfg<128, 128, 2, 2, false, false>(a, stream);
}

}  // namespace moeep
