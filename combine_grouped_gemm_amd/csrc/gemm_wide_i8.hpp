// Wide int8 grouped GEMM tile for experts with many rows (SwiGLU gate/up or
// plain down projection), used by ffn_i8.hip.
//
// A tile is up to BM rows of one expert by 256 weight rows (gate/up: 128 gate
// + 128 up rows of the same output columns, so the SwiGLU epilogue has g and u
// of a column in one wave).  A row's step of the contraction is 128 codes, the
// 128 bytes of a bf16 step, and v_mfma_i32_16x16x64_i8 takes the same 16 bytes
// per lane in the same layout as the bf16 instruction, so the operands move
// through the ring of gemm_wide.hpp: loads straight into LDS through bounded
// buffer resources, two stages, chunks XOR-swizzled by (row & 7), one copy of
// the k-loop per number of valid fragments, the weight stream two steps ahead.
// Half the bf16 kernel's bytes and instructions for the same product.
//
// The sums stay in int32 to the end: no scale touches the k-loop.  The tile's
// row and column scales are asked for before it and applied in the epilogue
// (row scales through LDS, a lane's column scales in registers).
#pragma once

#include "gemm_wide.hpp"

namespace moeep {
namespace widei8 {

using wide::block_barrier;
using wide::ic;
using wide::kNonTemporal;
using wide::kOutOfRange;
using wide::lds_addr;
using wide::lds_buf16;
using wide::lds_read16x4;
using wide::lds_read16x8;
using wide::make_rsrc;
using wide::rsrc_t;
using wide::swz;
using wide::wait_lgkm0;
using wide::wait_vmcnt;

typedef int intx4 __attribute__((ext_vector_type(4)));

constexpr int BN = 256;
constexpr int BK = 128;             // codes per k-step: 128 bytes per row
constexpr int CPR = 8;              // 16-byte chunks per row
constexpr int ROWB = 128;           // bytes per LDS row

// 8 waves laid out 2 (rows) x 4 (weight rows).  A wave owns the interleaved
// 16-row fragments {wm, wm + 2, ...} (so a short tile still spreads its valid
// rows over both row-waves) and 64 weight rows.
template <int BM, bool GATED, bool OUT_F32>
__global__ __launch_bounds__(512, 1) void grouped_gemm_i8_wide_kernel(FfnArgs p) {
    constexpr int WMW = 2, WNW = 4, NT = 512, NW = 8;
    constexpr int A_BLOCKS = BM * CPR / 64;          // 1 KiB blocks of a row stage
    constexpr int BLOCKS = (BM + BN) * CPR / 64;
    constexpr int LPS = BLOCKS / NW;                 // direct loads per wave per stage
    constexpr int FM = BM / 16 / WMW;                // 16-row fragments per wave
    constexpr int WN = BN / WNW;                     // 64 weight rows per wave
    constexpr int FN = WN / 16;                      // 4
    constexpr int BNO = GATED ? BN / 2 : BN;         // output columns per tile
    static_assert(BM % 32 == 0 && BLOCKS % NW == 0 && (!GATED || FN % 2 == 0), "tile shape");
    // block q = i * NW + wave: whether it is a row block and which weight half it
    // covers depends only on i, so both are compile-time after unrolling
    static_assert(A_BLOCKS % NW == 0 && (BN / 16) % NW == 0, "block split");
    constexpr int A_ITERS = A_BLOCKS / NW;           // i < A_ITERS: row blocks
    constexpr int G_ITERS = (BN / 16) / NW;          // next G_ITERS: gate (or first) weight half
    constexpr int B_ITERS = LPS - A_ITERS;           // weight loads per wave per stage
    // Tiles of at most 256 rows keep both k-halves' weight fragments of a step
    // in registers, so the weight buffer of step k takes step k + 2's weights
    // as soon as every wave holds them (the weight stream keeps up to two
    // steps in flight); 320-row tiles have no registers to spare for that.
    constexpr bool LOOK = BM <= 256;

    __shared__ uint4 sa0[BM * CPR];
    __shared__ uint4 sb0[BN * CPR];
    __shared__ uint4 sa1[BM * CPR];
    __shared__ uint4 sb1[BN * CPR];
    __shared__ int s_pre[kMaxExperts + 1];
    __shared__ uint16_t s_ord[kMaxExperts];          // experts, most rows first
    static_assert(sizeof(sa0) >= kMaxExperts * sizeof(int), "row counts fit in the first row stage");
    __shared__ int s_tmp[NT / kWave];
    __shared__ float s_as[BM];                       // the tile's row scales
    static_assert(BM <= NT, "one row scale per thread");

    auto a_base = [&](auto I) -> char* {
        if constexpr (decltype(I)::value == 0) return reinterpret_cast<char*>(sa0);
        else return reinterpret_cast<char*>(sa1);
    };
    auto b_base = [&](auto I) -> char* {
        if constexpr (decltype(I)::value == 0) return reinterpret_cast<char*>(sb0);
        else return reinterpret_cast<char*>(sb1);
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

    // largest experts' tiles first; the first row stage is free scratch until the first load
    build_tile_prefix_sorted<NT, BM>(p, s_pre, s_ord, reinterpret_cast<int*>(sa0), s_tmp);
    const int n_tiles_n = (N + BNO - 1) / BNO;
    const int total = n_tiles_n * s_pre[p.E_loc];
    const int G = gridDim.x;
    const int v = xcd_block_order();

    const uint8_t* __restrict__ A = static_cast<const uint8_t*>(p.a);
    const uint8_t* __restrict__ W0 = static_cast<const uint8_t*>(p.w0);
    const uint8_t* __restrict__ W1 = static_cast<const uint8_t*>(p.w1);

    for (int tau = v; tau < total; tau += G) {
        const TileCoord tc = decode_tile<BM>(tau, n_tiles_n, s_pre, p, s_ord);
        const int j = tc.j, row0 = tc.row0, nvalid = tc.nvalid;
        const int col0 = tc.nt * BNO;
        const uint8_t* wg = W0 + (size_t)j * N * ldw;
        const uint8_t* wu = GATED ? W1 + (size_t)j * N * ldw : nullptr;

        // Operands come in by buffer loads straight into LDS: a scalar resource
        // per operand (base, byte extent) plus a 32-bit per-lane offset and the
        // k-step as scalar offset.  Rows past the tile's valid rows and weight
        // rows past N lie outside their resource's extent, so those lanes read
        // nothing from memory and land zeros.  Each lane's offset is fixed for
        // the tile.
        const char* abase = reinterpret_cast<const char*>(A + (size_t)row0 * Kdim);
        const uint32_t a_bytes = (uint32_t)nvalid * (uint32_t)Kdim;
        const uint32_t w_bytes = (uint32_t)N * (uint32_t)ldw;
        uint32_t off[LPS];
#pragma unroll
        for (int i = 0; i < LPS; ++i) {
            const bool is_a = i < A_ITERS;
            const int r = (is_a ? i * NW : (i - A_ITERS) * NW) * 8 + wave * 8 + lane / 8;
            const uint32_t c16 = (uint32_t)swz(r, lane % 8) * 16;   // logical chunk this lane fetches
            const int rr = (!is_a && GATED && r >= BN / 2) ? r - BN / 2 : r;
            off[i] = (is_a ? (uint32_t)r * (uint32_t)Kdim : (uint32_t)(col0 + rr) * (uint32_t)ldw) + c16;
        }
        // direct load i of a stage; `live` false (the step after the last) reads
        // nothing, so every step issues the same LPS loads without a branch
        auto issue_one = [&](auto I, int i, int kstep, bool live) {
            const bool is_a = i < A_ITERS;
            const bool up = GATED && i >= A_ITERS + G_ITERS;
            char* dst = is_a ? a_base(I) + (i * NW + wave) * 1024
                             : b_base(I) + ((i - A_ITERS) * NW + wave) * 1024;
            // the step after the last gets an empty extent: every access out of range
            const rsrc_t r = make_rsrc(is_a ? (const void*)abase : (up ? (const void*)wu : (const void*)wg),
                                       live ? (is_a ? a_bytes : w_bytes) : 0u);
            // chunks past K (a partial last step) get an offset beyond every
            // extent, so they read nothing and land zeros in both operands
            const uint32_t vo = kstep * BK + lane_k < Kdim ? off[i] : kOutOfRange;
            // the row block is re-read by every n-tile of the expert (kept in
            // L2); weight tiles are read by one or two m-tiles close together in
            // tile order, so only the weights stream (non-temporal)
            if (is_a)
                lds_buf16<0>(r, dst, vo, kstep * BK);
            else
                lds_buf16<kNonTemporal>(r, dst, vo, kstep * BK);
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

        // the previous tile's reads of both stages must be complete before new loads land
        wait_lgkm0();
        block_barrier();
#pragma unroll
        for (int i = 0; i < LPS; ++i) issue_one(ic<0>{}, i, 0, true);
        {
            // and step 1's weights (nothing read when there is no step 1)
            const bool l1 = __builtin_amdgcn_readfirstlane(nk > 1 ? 1 : 0) != 0;
#pragma unroll
            for (int i = A_ITERS; i < LPS; ++i) issue_one(ic<1>{}, i, 1, l1);
        }

        // The tile for NF valid fragments: no branch inside a step.
        // v_mfma_i32_16x16x64_i8: lane l feeds row (l % 16) with k-chunk (l / 16)
        // of the 64-wide step for both operands and receives rows 4*(l/16)+e,
        // column l % 16 of the 16x16 result.
        auto tile = [&](auto NFc) {
            constexpr int NF = decltype(NFc)::value;
            intx4 acc[NF > 0 ? NF : 1][FN];
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int f = 0; f < FN; ++f) acc[i][f] = intx4{0, 0, 0, 0};

            // LOOK: read both k-halves' weight fragments of step k, and once every
            // wave holds them issue, one after each fragment's MFMA group, step
            // k + 1's row loads into the other row buffer and then step k + 2's
            // weight loads into this step's weight buffer (loads past the last
            // step read nothing but count, so every step issues LPS loads)
            auto compute_look = [&](auto I, int k, bool liveA, bool liveB) {
                const char* ab = a_base(I);
                const char* bb = b_base(I);
                constexpr auto nextbuf = ic<1 - decltype(I)::value>{};
                static_assert(2 * FN == 8, "weight fragment reads");
                intx4 bfr[2][FN];
                {
                    uint32_t ad[8];
                    uint4 t[8];
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                        for (int f = 0; f < FN; ++f) ad[kk * FN + f] = lds_addr(bb + lds_lane[kk] + brow0(f) * ROWB);
                    lds_read16x8(t, ad);
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                        for (int f = 0; f < FN; ++f) bfr[kk][f] = __builtin_bit_cast(intx4, t[kk * FN + f]);
                }
                block_barrier();
                auto issue_slot = [&](int q) {
                    if (q < A_ITERS) issue_one(nextbuf, q, k + 1, liveA);
                    else issue_one(I, q, k + 2, liveB);
                };
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    intx4 acur;
                    if (NF > 0) acur = *reinterpret_cast<const intx4*>(ab + lds_lane[kk] + wm * 16 * ROWB);
#pragma unroll
                    for (int i = 0; i < NF; ++i) {
                        intx4 anext;
                        if (i + 1 < NF)
                            anext = *reinterpret_cast<const intx4*>(
                                ab + lds_lane[kk] + (wm + WMW * (i + 1)) * 16 * ROWB);
#pragma unroll
                        for (int f = 0; f < FN; ++f)
                            acc[i][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(acur, bfr[kk][f], acc[i][f], 0, 0, 0);
                        const int slot = kk * NF + i;
                        if (slot < LPS) issue_slot(slot);
                        if (i + 1 < NF) acur = anext;
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                if (2 * NF < LPS) {
#pragma unroll
                    for (int q = 2 * NF; q < LPS; ++q) issue_slot(q);
                }
            };

            // !LOOK: the first k-half issues step k + 1's row
            // loads and the second half, once every wave holds its weight
            // fragments, step k + 2's weight loads into this step's buffer
            auto compute_half = [&](auto I, int k, bool liveA, bool liveB) {
                const char* ab = a_base(I);
                const char* bb = b_base(I);
                constexpr auto nextbuf = ic<1 - decltype(I)::value>{};
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    intx4 bfr[FN];
                    {
                        static_assert(FN == 4, "weight fragment reads");
                        uint32_t ad[4];
                        uint4 t[4];
#pragma unroll
                        for (int f = 0; f < FN; ++f) ad[f] = lds_addr(bb + lds_lane[kk] + brow0(f) * ROWB);
                        lds_read16x4(t, ad);
#pragma unroll
                        for (int f = 0; f < FN; ++f) bfr[f] = __builtin_bit_cast(intx4, t[f]);
                    }
                    if (kk == 1) block_barrier();      // every wave holds this step's weight fragments
                    intx4 acur;
                    if (NF > 0) acur = *reinterpret_cast<const intx4*>(ab + lds_lane[kk] + wm * 16 * ROWB);
#pragma unroll
                    for (int i = 0; i < NF; ++i) {
                        intx4 anext;
                        if (i + 1 < NF)
                            anext = *reinterpret_cast<const intx4*>(
                                ab + lds_lane[kk] + (wm + WMW * (i + 1)) * 16 * ROWB);
#pragma unroll
                        for (int f = 0; f < FN; ++f)
                            acc[i][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(acur, bfr[f], acc[i][f], 0, 0, 0);
                        if (kk == 0 && i < A_ITERS) issue_one(nextbuf, i, k + 1, liveA);
                        if (kk == 1 && i < B_ITERS) issue_one(I, A_ITERS + i, k + 2, liveB);
                        if (i + 1 < NF) acur = anext;
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if (kk == 0 && NF < A_ITERS) {
#pragma unroll
                        for (int q = NF; q < A_ITERS; ++q) issue_one(nextbuf, q, k + 1, liveA);
                    }
                    if (kk == 1 && NF < B_ITERS) {
#pragma unroll
                        for (int q = NF; q < B_ITERS; ++q) issue_one(I, A_ITERS + q, k + 2, liveB);
                    }
                }
            };

            // step k: wait for stage k (step k + 1's weights stay in flight), then
            // compute k while stage k + 1 is loaded into the other buffer
            auto step = [&](auto I, int k) {
                wait_vmcnt<B_ITERS>();
                wait_lgkm0();
                block_barrier();
                // wave-uniform by construction; say so, so that the resource
                // select below stays scalar
                const bool live = __builtin_amdgcn_readfirstlane(k + 1 < nk ? 1 : 0) != 0;
                const bool live2 = __builtin_amdgcn_readfirstlane(k + 2 < nk ? 1 : 0) != 0;
                if constexpr (LOOK) compute_look(I, k, live, live2);
                else compute_half(I, k, live, live2);
            };
            for (int k = 0; k < nk; k += 2) {
                step(ic<0>{}, k);
                if (k + 1 < nk) step(ic<1>{}, k + 1);
            }
            // the loads issued by the last step read nothing but still count
            wait_vmcnt<0>();

            // ---- epilogue: every wave stages its outputs in a private LDS region
            // (both stages are free once every wave is past the k-loop) and
            // stores whole 16-byte row chunks.  PF fragments per pass; staged
            // rows are padded by 16 bytes so that the four row groups of one LDS
            // write fall into different banks.
            constexpr int OSZ = OUT_F32 ? 4 : 2;            // bytes per output
            constexpr int OCOLS = FO * 16;                  // output columns of a wave
            constexpr int OCH = OCOLS * OSZ / 16;           // 16-byte chunks per staged row
            constexpr int OPITCH = OCOLS * OSZ + 16;        // staged row pitch (bytes)
            constexpr int PF = OUT_F32 ? 3 : 5;             // fragments per pass
            constexpr int RSZ = PF * 16 * OPITCH;           // bytes of a wave's region
            static_assert(2 * RSZ <= BN * ROWB && 2 * RSZ <= BM * ROWB, "two regions per stage buffer");
            if (tid < BM) s_as[tid] = row_s;
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
                        const float4 rs = *reinterpret_cast<const float4*>(s_as + (wm + WMW * i) * 16 + (lane >> 4) * 4);
                        const float rse[4] = {rs.x, rs.y, rs.z, rs.w};
#pragma unroll
                        for (int f = 0; f < FO; ++f)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float val = (float)acc[i][f][e] * rse[e] * col_s[f];
                                if constexpr (GATED)
                                    val = silu(val) * ((float)acc[i][f + FO][e] * rse[e] * col_s[f + FO]);
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
        static_assert(FM <= 10, "one case per fragment count");
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
            case 9: if constexpr (9 <= FM) tile(ic<9>{}); break;
            case 10: if constexpr (10 <= FM) tile(ic<10>{}); break;
            default: break;
        }
    }
}

}  // namespace widei8
}  // namespace moeep
