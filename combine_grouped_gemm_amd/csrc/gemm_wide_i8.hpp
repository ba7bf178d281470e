// Int8 grouped GEMM tile (SwiGLU gate/up or plain down projection), used by
// ffn_i8.hip.
//
// A tile is up to BM rows of one expert by BN weight rows (gate/up: BN / 2
// gate + BN / 2 up rows of the same output columns, so the SwiGLU epilogue has
// g and u of a column in one wave).  A row's step of the contraction is 128
// codes, one cache line; v_mfma_i32_16x16x64_i8 takes 16 bytes per lane of
// each operand.  Operands go from global memory straight into LDS through
// bounded buffer resources, in S stages (two; three where two workgroups of
// them fit a CU); the 16-byte chunks of an LDS row are XOR-swizzled by (row &
// 7), so the rows of one MFMA operand read fall into distinct banks; a tile
// runs one of FM + 1 copies of the k-loop by its count of valid row fragments
// (as gemm_wide.hpp does, with which it shares the load and wait helpers).
//
// Where it differs is what is in flight.  The second k-half's fragments are
// read under the first half's MFMAs, so that half-way through step k every
// wave holds all it needs of the stage, rows and weights alike, and step
// k + S's loads go into it: S - 1/2 steps ahead for both operands.
// With the weights ahead but the rows only one step (the bf16 scheme) every
// step waited for its rows' first touch of the XCD's L2.
//
// The sums stay in int32 to the end: no scale touches the k-loop.  The tile's
// row and column scales are asked for before it and applied in the epilogue
// (row scales through LDS, a lane's column scales in registers).
//
// Measured (MI355X, several boxes; DeepSeek-shaped layer, H = 7168, I = 2048,
// 256 experts): decode gate/up, T = 128: 0.97-0.99 ms, 6.7-6.9 TB/s (some 230 of
// the experts have a row; counters: 6.68 GB in 969 us; two stages 977); down 0.55-
// 0.56 ms, 6.1 TB/s (two stages 0.56).  One token (8 experts): 39 us, 6.0 TB/s.
// One EP=8 rank's share: 0.21-0.22 ms, 4.4-4.7 TB/s at a 2.25 GHz clock, the CUs
// busy three quarters of the time (2.2 tiles each, of unequal sizes).  Prefill,
// T = 8192: 2.1-2.3 ms, 1.7-1.8 POP/s; counters show the MFMAs busy 54% of the
// cycles at a clock of 1.4 GHz, and versions with 10% fewer cycles took the same
// time: the part's power holds it there (MFMAs alone, fed from registers, reach
// 4.2 POP/s; the 32x32x32 form 3.6).  Four waves of 128 x 128 instead of eight
// of 128 x 64, which read a third less LDS, spill and take 2.6 ms.
// 256 x 256 with fp32 outputs uses all 256 VGPRs and 36 bytes of scratch a lane;
// the reloads lie outside the k-loop and cannot be seen: 256 experts of 256 rows,
// down at H = 7168, 1375 us against 1239 with bf16 outputs, less than the 0.94 GB
// more that are written take in a copy.
#pragma once

#include "gemm_wide.hpp"

namespace moeep {
namespace widei8 {

using wide::block_barrier;
using wide::ic;
using wide::kNonTemporal;
using wide::kOutOfRange;
using wide::lds_buf16;
using wide::make_rsrc;
using wide::rsrc_t;
using wide::swz;
using wide::wait_lgkm0;
using wide::wait_vmcnt;

typedef int intx4 __attribute__((ext_vector_type(4)));

constexpr int BK = 128;             // codes per k-step: 128 bytes per row
constexpr int CPR = 8;              // 16-byte chunks per row
constexpr int ROWB = 128;           // bytes per LDS row

// An output is acc * row scale * channel scale.  In that order alone rows of
// 1e33 and more (scale: amax / 127) made infinities of finite results.  The row
// scale r is therefore split into r1 = r, r2 = 1 where |r| < 1 and r1 = 1, r2 = r
// elsewhere, and the product is ((acc r1) c) r2: one factor is 1, so there are
// two roundings still.  Nothing overflows on the way to a result P that fp32
// holds: |acc r1| <= 2^31, (acc r) c = P or |acc c| = |P / r| <= |P|.  Nor is
// anything lost at fp32's start: |acc| >= 1 keeps the first product at or above
// a scale, and one below 2^-126 is a whole multiple of 2^-149.  A NaN compares
// false and stays in r2.  (Within 0.4% of two products; choosing the order for
// each output, a compare and two selects, took 1% more in down at 2880.)
__device__ __forceinline__ float scaled(int acc, float r1, float c, float r2) { return (float)acc * r1 * c * r2; }

// silu with its limit, zero, where g lies below fp32's range (-inf * 0 is NaN).
// The maximum keeps a NaN, in one instruction (v_maximum3_f32).
__device__ __forceinline__ float silu_finite(float g) {
    return silu(__builtin_elementwise_maximum(g, -3.40282347e38f));
}

// 8 waves laid out 2 (rows) x 4 (weight rows).  A wave owns the interleaved
// 16-row fragments {wm, wm + 2, ...} (so a short tile still spreads its valid
// rows over both row-waves) and BN / 4 weight rows.  S: stages, 2 or 3.
template <int BM, int BN, int S, bool GATED, bool OUT_F32, bool NT_W>
__global__ __launch_bounds__(512, BM + BN > 256 ? 1 : 4) void grouped_gemm_i8_wide_kernel(FfnArgs p) {
    constexpr int WMW = 2, WNW = 4, NT = 512, NW = 8;
    constexpr int A_BLOCKS = BM * CPR / 64;          // 1 KiB blocks of a row stage
    constexpr int BLOCKS = (BM + BN) * CPR / 64;
    constexpr int LPS = BLOCKS / NW;                 // direct loads per wave per stage
    constexpr int FM = BM / 16 / WMW;                // 16-row fragments per wave
    constexpr int WN = BN / WNW;                     // weight rows per wave
    constexpr int FN = WN / 16;                      // 16-row weight fragments per wave
    constexpr int BNO = GATED ? BN / 2 : BN;         // output columns per tile
    static_assert((S == 2 || S == 3) && BM % 32 == 0 && BLOCKS % NW == 0 && (!GATED || FN % 2 == 0), "tile shape");
    constexpr int A_ITERS = A_BLOCKS / NW;           // i < A_ITERS: row blocks
    constexpr int RPL = NW * 8;                      // operand rows that one load of every wave covers
    constexpr int G_ITERS = BN / 2 / RPL;            // next G_ITERS: the gate half
    // whether a load's rows are token rows, and which weight half they belong to,
    // is compile-time after unrolling
    static_assert(BM % RPL == 0 && BN / 2 % RPL == 0, "whole loads");

    __shared__ uint4 sa0[BM * CPR];
    __shared__ uint4 sb0[BN * CPR];
    __shared__ uint4 sa1[BM * CPR];
    __shared__ uint4 sb1[BN * CPR];
    __shared__ uint4 sa2[S > 2 ? BM * CPR : 1];
    __shared__ uint4 sb2[S > 2 ? BN * CPR : 1];
    __shared__ int s_pre[kMaxExperts + 1];
    // experts, most rows first.  Small tiles keep the experts' own order: theirs are
    // nearly all alike (weights, whatever the rows), and ranking 256 experts takes
    // 7 us (one token at H = 7168 46.4 us with it, 39.1 without; 16 tokens 473, 435;
    // decode down 562, 553).
    constexpr bool SORTED = BM > 64;
    __shared__ uint16_t s_ord[SORTED ? kMaxExperts : 1];
    static_assert(sizeof(sa0) >= kMaxExperts * sizeof(int), "row counts fit in the first row stage");
    __shared__ int s_tmp[NT / kWave];
    __shared__ float s_as[2][BM];                    // the tile's row scales, split (see scaled)
    static_assert(BM <= NT, "one row scale per thread");

    auto a_base = [&](auto I) -> char* {
        if constexpr (decltype(I)::value == 0) return reinterpret_cast<char*>(sa0);
        else if constexpr (decltype(I)::value == 1) return reinterpret_cast<char*>(sa1);
        else return reinterpret_cast<char*>(sa2);
    };
    auto b_base = [&](auto I) -> char* {
        if constexpr (decltype(I)::value == 0) return reinterpret_cast<char*>(sb0);
        else if constexpr (decltype(I)::value == 1) return reinterpret_cast<char*>(sb1);
        else return reinterpret_cast<char*>(sb2);
    };

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);   // uniform: keeps LDS bases scalar
    const int wm = wave / WNW, wn = wave % WNW;
    const int Kdim = p.Kdim, N = p.N;
    const int ldw = p.ldw;                          // weight row pitch (bytes)
    const int nk = (Kdim + BK - 1) / BK;            // the last k-step may be partial (K % 128 != 0)
    // contraction offset, within a k-step, of the 16-byte chunk this lane
    // fetches in every direct load (rows of a load's 1 KiB block start at
    // multiples of 8, so a row's (row & 7) is lane / 8)
    const int lane_k = swz(lane / 8, lane % 8) * 16;

    // the first row stage is free scratch until the first load
    if constexpr (SORTED) build_tile_prefix_sorted<NT, BM>(p, s_pre, s_ord, reinterpret_cast<int*>(sa0), s_tmp);
    else build_tile_prefix<NT, BM>(p, s_pre, s_tmp);
    const int n_tiles_n = (N + BNO - 1) / BNO;
    const int total = n_tiles_n * s_pre[p.E_loc];
    const int G = gridDim.x;
    const int v = xcd_block_order();

    const uint8_t* __restrict__ A = static_cast<const uint8_t*>(p.a);
    const uint8_t* __restrict__ W0 = static_cast<const uint8_t*>(p.w0);
    const uint8_t* __restrict__ W1 = static_cast<const uint8_t*>(p.w1);

    // Large tiles come in order of decreasing cost: every other round runs backwards
    // over the blocks, so that none gets the largest tile of every round.  A round that
    // fills less than three quarters of the grid goes in hardware order, over all
    // XCDs; in XCD-major order it would leave some of them idle (one token's 8
    // experts, gate/up at H = 7168: 69.7 -> 44.7 us; 16 tokens 476 -> 454).  Large
    // tiles do so only if it is their one round: in a last round after others
    // sharing rows in an XCD's L2 is worth more (EP share 224 us, 228 spread).
    for (int base = 0, rnd = 0; base < total; base += G, ++rnd) {
        const bool sparse = (BM < 256 || rnd == 0) && (long long)(total - base) * 4 < (long long)G * 3;
        const int at = sparse ? (int)blockIdx.x : v;
        const int tau = base + (rnd & 1 ? G - 1 - at : at);
        if (tau >= total) continue;
        const TileCoord tc = decode_tile<BM>(tau, n_tiles_n, s_pre, p, SORTED ? s_ord : nullptr);
        const int j = tc.j, row0 = tc.row0, nvalid = tc.nvalid;
        const int col0 = tc.nt * BNO;
        // the tile's weight rows start at output column col0
        const size_t w0 = ((size_t)j * N + col0) * ldw;
        const uint8_t* wg = W0 + w0;
        const uint8_t* wu = GATED ? W1 + w0 : nullptr;

        // Operands come in by buffer loads straight into LDS: a scalar resource
        // (base, byte extent) per operand, the k-step as scalar offset and a
        // 32-bit lane offset, the row's.  Rows past the tile's valid rows and
        // weight rows past N lie outside their resource's extent, so those lanes
        // read nothing from memory and land zeros.
        const uint8_t* abase = A + (size_t)row0 * Kdim;
        const uint32_t a_bytes = (uint32_t)nvalid * (uint32_t)Kdim;
        const uint32_t w_bytes = (uint32_t)min(N - col0, BNO) * (uint32_t)ldw;   // of the tile (of each half)
        const uint32_t lrow = wave * 8 + lane / 8;              // this lane's row of a load's RPL rows
        const uint32_t off_a = lrow * (uint32_t)Kdim + lane_k, off_w = lrow * (uint32_t)ldw + lane_k;
        // direct load i of a stage; `live` false (a step past the last) reads
        // nothing, so every step issues the same LPS loads without a branch
        auto issue_one = [&](auto I, int i, int kstep, bool live) {
            const bool is_a = i < A_ITERS;
            const int q = i - A_ITERS;                          // RPL-row block of the weights
            const bool up = GATED && q >= G_ITERS;
            const int first = is_a ? i * RPL : (up ? q - G_ITERS : q) * RPL;
            char* dst = is_a ? a_base(I) + (i * NW + wave) * 1024 : b_base(I) + (q * NW + wave) * 1024;
            const rsrc_t r = make_rsrc(is_a ? abase : up ? wu : wg, live ? (is_a ? a_bytes : w_bytes) : 0u);
            // chunks past K (a partial last step) get an offset beyond every
            // extent, so they read nothing and land zeros in both operands
            // (formed anew for every load: kept in registers from step to step, the
            // offsets push accumulators out to memory)
            uint32_t down = (uint32_t)first * (uint32_t)(is_a ? Kdim : ldw);
            asm volatile("" : "+s"(down));
            const uint32_t row = (is_a ? off_a : off_w) + down;
            const uint32_t vo = kstep * BK + lane_k < Kdim ? row : kOutOfRange;
            // the row block is re-read by every n-tile of the expert (kept in
            // L2); the weights' cache policy is the launcher's choice
            if (is_a)
                lds_buf16<0>(r, dst, vo, kstep * BK);
            else
                lds_buf16<NT_W ? kNonTemporal : 0>(r, dst, vo, kstep * BK);
        };

        // per-lane LDS byte offset of the 16-byte chunk this lane feeds to an
        // MFMA at half-step kk, for any operand row that is a multiple of 16
        // plus (lane & 15): the swizzle then depends on the lane alone
        int lds_lane[2];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
            lds_lane[kk] = (lane & 15) * ROWB + (((kk * 4 + (lane >> 4)) ^ (lane & 7)) * 16);
        auto brow0 = [&](int f) {     // first B-tile row of n-fragment f
            if (GATED) {
                const int half = f < FN / 2 ? 0 : BN / 2;
                const int ff = f < FN / 2 ? f : f - FN / 2;
                return half + wn * (WN / 2) + ff * 16;
            }
            return wn * WN + f * 16;
        };
        auto fcol = [&](int f) {      // output column of fragment f's first lane column
            if (GATED) {
                const int ff = f < FN / 2 ? f : f - FN / 2;
                return col0 + wn * (WN / 2) + ff * 16;
            }
            return col0 + wn * WN + f * 16;
        };

        // this wave's valid 16-row fragments are i < nf (rows (wm + 2 i) * 16 ...)
        const int nf = __builtin_amdgcn_readfirstlane(
            nvalid > wm * 16 ? min(FM, (nvalid - wm * 16 + 31) / 32) : 0);

        // the scales of the epilogue, asked for before the k-loop: this thread's
        // row (through LDS later) and this lane's output columns
        constexpr int FO = GATED ? FN / 2 : FN;
        float row_s = 0.0f;
        if (tid < nvalid) row_s = p.a_scales[row0 + tid];
        float col_s[FN];
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            const int col = fcol(f) + (lane & 15);
            const float* s = GATED && f >= FO ? p.w1_scales : p.w0_scales;
            col_s[f] = col < N ? s[(size_t)j * N + col] : 0.0f;
        }

        // the previous tile's reads of the stages must be complete before new loads land
        wait_lgkm0();
        block_barrier();
        // steps 0 .. S - 1 (nothing read for a step that does not exist)
        auto fill = [&](auto I) {
            const bool exists = __builtin_amdgcn_readfirstlane(decltype(I)::value < nk ? 1 : 0) != 0;
#pragma unroll
            for (int i = 0; i < LPS; ++i) issue_one(I, i, decltype(I)::value, exists);
        };
        fill(ic<0>{});
        fill(ic<1>{});
        if constexpr (S > 2) fill(ic<2>{});

        // The tile for NF valid fragments: no branch inside a step.
        // v_mfma_i32_16x16x64_i8: lane l feeds row (l % 16) with k-chunk (l / 16)
        // of the 64-wide step for both operands and receives rows 4*(l/16)+e,
        // column l % 16 of the 16x16 result.
        auto tile = [&](auto NFc) {
            constexpr int NF = decltype(NFc)::value, NG = NF > 0 ? NF : 1;
            intx4 acc[NG][FN];
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int f = 0; f < FN; ++f) acc[i][f] = intx4{0, 0, 0, 0};

            // Step k out of stage I.  The second k-half's fragments are read under
            // the first half's MFMAs; once every wave holds them the stage is
            // free, rows and weights alike, and step k + S's loads go into it
            // between the second half's MFMA groups (loads past the last step
            // read nothing but count).
            auto compute = [&](auto I, int k, bool live) {
                const char* ab = a_base(I) + wm * 16 * ROWB;
                const char* bb = b_base(I);
                auto read_a = [&](int kk, int i) {
                    return *reinterpret_cast<const intx4*>(ab + lds_lane[kk] + i * WMW * 16 * ROWB);
                };
                auto read_b = [&](int kk, int f) {
                    return *reinterpret_cast<const intx4*>(bb + lds_lane[kk] + brow0(f) * ROWB);
                };
                intx4 af[2][NG], bf[2][FN];
                if (NF > 0) {
#pragma unroll
                    for (int f = 0; f < FN; ++f) bf[0][f] = read_b(0, f);
#pragma unroll
                    for (int i = 0; i < NF; ++i) af[0][i] = read_a(0, i);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < NF; ++i) {
#pragma unroll
                    for (int f = 0; f < FN; ++f)
                        acc[i][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[0][i], bf[0][f], acc[i][f], 0, 0, 0);
                    if (i == 0) {
#pragma unroll
                        for (int f = 0; f < FN; ++f) bf[1][f] = read_b(1, f);
                    }
                    af[1][i] = read_a(1, i);
                    __builtin_amdgcn_sched_barrier(0);
                }
                wait_lgkm0();
                block_barrier();
#pragma unroll
                for (int i = 0; i < NF; ++i) {
#pragma unroll
                    for (int f = 0; f < FN; ++f)
                        acc[i][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[1][i], bf[1][f], acc[i][f], 0, 0, 0);
#pragma unroll
                    for (int q = i * LPS / NG; q < (i + 1) * LPS / NG; ++q) issue_one(I, q, k + S, live);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (NF == 0) {
#pragma unroll
                    for (int q = 0; q < LPS; ++q) issue_one(I, q, k + S, live);
                }
            };

            // step k: wait for its stage (the S - 1 later ones stay in flight)
            auto step = [&](auto I, int k) {
                wait_vmcnt<(S - 1) * LPS>();
                block_barrier();
                // wave-uniform by construction; say so, so that the resource
                // select below stays scalar
                const bool live = __builtin_amdgcn_readfirstlane(k + S < nk ? 1 : 0) != 0;
                compute(I, k, live);
            };
            // S steps a turn without a branch between them: with one, the compiler no
            // longer knew which loads were in flight at the top of the loop and waited
            // for all of them there
            int k = 0;
            for (; k + S - 1 < nk; k += S) {
                step(ic<0>{}, k);
                step(ic<1>{}, k + 1);
                if constexpr (S > 2) step(ic<2>{}, k + 2);
            }
            if (k < nk) step(ic<0>{}, k);
            if constexpr (S > 2) {
                if (k + 1 < nk) step(ic<1>{}, k + 1);
            }
            // the loads issued by the last step read nothing but still count
            wait_vmcnt<0>();

            // ---- epilogue: every wave stages its outputs in a private LDS region
            // (the stages are free once every wave is past the k-loop) and
            // stores whole 16-byte row chunks.  PF fragments per pass; staged
            // rows are padded by 16 bytes so that the four row groups of one LDS
            // write fall into different banks.
            constexpr int OSZ = OUT_F32 ? 4 : 2;            // bytes per output
            constexpr int OCOLS = FO * 16;                  // output columns of a wave
            constexpr int OCH = OCOLS * OSZ / 16;           // 16-byte chunks per staged row
            constexpr int OPITCH = OCOLS * OSZ + 16;        // staged row pitch (bytes)
            constexpr int PF_MAX = (BM < BN ? BM : BN) * ROWB / 2 / (16 * OPITCH);
            constexpr int PF = PF_MAX < FM ? PF_MAX : FM;   // fragments per pass
            constexpr int RSZ = PF * 16 * OPITCH;           // bytes of a wave's region
            static_assert(PF >= 1 && 2 * RSZ <= BN * ROWB && 2 * RSZ <= BM * ROWB, "two regions per stage buffer");
            if (tid < BM) {
                const bool below = fabsf(row_s) < 1.0f;
                s_as[0][tid] = below ? row_s : 1.0f;
                s_as[1][tid] = below ? 1.0f : row_s;
            }
            wait_lgkm0();
            block_barrier();
            char* region = (wave < 2 ? reinterpret_cast<char*>(sa0) : wave < 4 ? reinterpret_cast<char*>(sb0)
                            : wave < 6 ? reinterpret_cast<char*>(sa1) : reinterpret_cast<char*>(sb1)) + (wave & 1) * RSZ;
            const int colbase = fcol(0);                    // the wave's first output column
            char* out_bytes = static_cast<char*>(p.out);
#pragma unroll
            for (int p0 = 0; p0 < NF; p0 += PF) {
#pragma unroll
                for (int ii = 0; ii < PF; ++ii) {
                    const int i = p0 + ii;
                    if (i < NF) {
                        const int r4 = (wm + WMW * i) * 16 + (lane >> 4) * 4;
                        const float4 v1 = *reinterpret_cast<const float4*>(s_as[0] + r4);
                        const float4 v2 = *reinterpret_cast<const float4*>(s_as[1] + r4);
                        const float r1[4] = {v1.x, v1.y, v1.z, v1.w}, r2[4] = {v2.x, v2.y, v2.z, v2.w};
#pragma unroll
                        for (int f = 0; f < FO; ++f)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float val = scaled(acc[i][f][e], r1[e], col_s[f], r2[e]);
                                if constexpr (GATED)
                                    val = silu_finite(val) * scaled(acc[i][f + FO][e], r1[e], col_s[f + FO], r2[e]);
                                char* at = region + (ii * 16 + (lane >> 4) * 4 + e) * OPITCH + (f * 16 + (lane & 15)) * OSZ;
                                if constexpr (OUT_F32) *reinterpret_cast<float*>(at) = val;
                                else *reinterpret_cast<uint16_t*>(at) = (uint16_t)f32_to_bf16_bits(val);
                            }
                    }
                }
                constexpr int RPI = 64 / OCH;               // staged rows per 64-lane read
#pragma unroll
                for (int q = 0; q < PF * 16 / RPI; ++q) {
                    const int lrow = q * RPI + lane / OCH, ch = lane % OCH;
                    const int i = p0 + lrow / 16;
                    const int trow = (wm + WMW * i) * 16 + lrow % 16;   // row within the tile
                    const int col = colbase + ch * (16 / OSZ);
                    if (i < NF && trow < nvalid && col < N) {
                        const uint4 v = *reinterpret_cast<const uint4*>(region + lrow * OPITCH + ch * 16);
                        *reinterpret_cast<uint4*>(out_bytes + ((size_t)(row0 + trow) * N + col) * OSZ) = v;
                    }
                }
            }
        };
        // a switch, not a chain of ifs: with the chain the compiler no longer
        // treated the tile's scalars as uniform and wrapped every buffer load
        // in a readfirstlane loop
        static_assert(FM <= 8, "one case per fragment count");
        switch (nf) {
            case 0: if constexpr (0 <= FM) tile(ic<0>{}); break;
            case 1: if constexpr (1 <= FM) tile(ic<1>{}); break;
            case 2: if constexpr (2 <= FM) tile(ic<2>{}); break;
            case 3: if constexpr (3 <= FM) tile(ic<3>{}); break;
            case 4: if constexpr (4 <= FM) tile(ic<4>{}); break;
            case 5: if constexpr (5 <= FM) tile(ic<5>{}); break;
            case 6: if constexpr (6 <= FM) tile(ic<6>{}); break;
            case 7: if constexpr (7 <= FM) tile(ic<7>{}); break;
            case 8: if constexpr (8 <= FM) tile(ic<8>{}); break;
            default: break;
        }
    }
}

}  // namespace widei8
}  // namespace moeep
