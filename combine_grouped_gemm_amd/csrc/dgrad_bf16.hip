// Input gradients of the grouped products in bf16: dx[r] = dy[r] W_j (+ dy2[r] W2_j)
// for the rows of every local expert, fp32 accumulation on MFMA.
//
// The forward kernels' tiles and rings (gemm_wide.hpp, ffn_bf16.hip) with the weights
// contracted over their rows: a k-step of W is 64 rows of the tile's columns, and its
// fragments are transposing LDS reads (gemm_cols.hpp).  A pair of products is one k-loop
// that goes through both.  With src_of a row of dy is looked up once per tile: every
// direct load has its own per-lane row offset anyway, so the gather costs the loop
// nothing and the dispatched copy of dy is never made.
#include "gemm_cols.hpp"

namespace moeep {
namespace {

using namespace cols;

// row of dy that expert row r reads (-1: none)
__device__ __forceinline__ int dy_row(const FfnArgs& p, int r) {
    if (p.src_of == nullptr) return r;
    const int s = p.src_of[r];
    if (s < 0) return -1;
    const int t = token_of(s, p.per_div);
    return t < p.src_rows ? t : -1;
}

// ---- row-rich experts: 8 waves 2 (rows) x 4 (columns), tiles of up to BM rows by 256
// columns, two-stage ring.  Tiles of at most 256 rows keep both halves' weight fragments
// of a step in registers and so release its weight stage to step k + 2 at once; 320-row
// tiles release it half-way (gemm_wide.hpp has the reasons and what they measured).
template <int BM>
__global__ __launch_bounds__(512, 1) void dgrad_wide_kernel(FfnArgs p) {
    constexpr int WMW = 2, WNW = 4, NT = 512, NW = 8;
    constexpr int A_ITERS = BM * CPR / 64 / NW;      // row loads of a wave per stage
    constexpr int B_ITERS = BK * BN * 2 / 1024 / NW; // weight loads: 1 KiB is two rows of 256 columns
    constexpr int LPS = A_ITERS + B_ITERS;
    constexpr int FM = BM / 16 / WMW, FN = BN / WNW / 16;
    constexpr bool LOOK = BM <= 256;
    static_assert(BM % 64 == 0 && B_ITERS == 4 && FN == 4, "tile shape");

    __shared__ uint4 sa0[BM * CPR];
    __shared__ uint4 sb0[BK * BN / 8];
    __shared__ uint4 sa1[BM * CPR];
    __shared__ uint4 sb1[BK * BN / 8];
    __shared__ int s_pre[kMaxExperts + 1];
    __shared__ uint16_t s_ord[kMaxExperts];
    static_assert(sizeof(sa0) >= kMaxExperts * sizeof(int), "row counts fit in the first row stage");
    __shared__ int s_tmp[NT / kWave];

    auto a_base = [&](auto I) -> char* {
        if constexpr (decltype(I)::value == 0) return reinterpret_cast<char*>(sa0);
        else return reinterpret_cast<char*>(sa1);
    };
    auto b_base = [&](auto I) -> char* {
        if constexpr (decltype(I)::value == 0) return reinterpret_cast<char*>(sb0);
        else return reinterpret_cast<char*>(sb1);
    };

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / WNW, wn = wave % WNW;
    const int Kdim = p.Kdim, N = p.N, ldw = p.ldw;
    const int nk1 = (Kdim + BK - 1) / BK, nk = p.a2 != nullptr ? 2 * nk1 : nk1;
    const int lane_k = swz(lane / 8, lane % 8) * 8;

    build_tile_prefix_sorted<NT, BM, true>(p, s_pre, s_ord, reinterpret_cast<int*>(sa0), s_tmp);
    const int n_tiles_n = (N + BN - 1) / BN;
    const int total = n_tiles_n * s_pre[p.E_loc];
    const int G = gridDim.x;
    const int v = xcd_block_order();
    uint16_t* __restrict__ Out = static_cast<uint16_t*>(p.out);

    for (int rnd = 0; rnd * (long long)G < total; ++rnd) {
        const int tau = round_tile_back(rnd, v, G, total);
        if (tau < 0) continue;                           // (an odd last round fills from the other end)
        const TileCoord tc = decode_tile<BM>(tau, n_tiles_n, s_pre, p, s_ord);
        const int j = tc.j, row0 = tc.row0, nvalid = tc.nvalid;
        const int col0 = tc.nt * BN;

        // Lane offsets, fixed for the tile.  Row loads: rows of dy relative to the tile's
        // first row, or anywhere in dy; a row past the tile's, or one that src_of names
        // nowhere, is out of range and lands zeros.  Weight loads: relative to the step's
        // first row, whose address and extent (rows left, so that rows past the last read
        // nothing) move with the step; columns past N are out of range.
        const size_t first = p.src_of != nullptr ? 0 : (size_t)row0 * Kdim;
        const char* abase[2] = {reinterpret_cast<const char*>(static_cast<const uint16_t*>(p.a) + first),
                                reinterpret_cast<const char*>(static_cast<const uint16_t*>(p.a2) + first)};
        const uint32_t a_bytes = (uint32_t)(p.src_of != nullptr ? p.src_rows : nvalid) * (uint32_t)(Kdim * 2);
        const char* wbase[2] = {reinterpret_cast<const char*>(static_cast<const uint16_t*>(p.w0) + (size_t)j * Kdim * ldw),
                                reinterpret_cast<const char*>(static_cast<const uint16_t*>(p.w1) + (size_t)j * Kdim * ldw)};
        uint32_t off[LPS];
#pragma unroll
        for (int i = 0; i < LPS; ++i) {
            if (i < A_ITERS) {
                const int r = (i * NW + wave) * 8 + lane / 8;
                int q = -1;
                if (r < nvalid) q = p.src_of != nullptr ? dy_row(p, row0 + r) : r;
                off[i] = q >= 0 ? (uint32_t)q * (uint32_t)(Kdim * 2) + (uint32_t)swz(r, lane % 8) * 16 : kOutOfRange;
            } else {
                const int k = ((i - A_ITERS) * NW + wave) * 2 + lane / 32;
                const int c = (lane % 32) ^ swz_row<BN>(k);
                off[i] = col0 + c * 8 < N ? (uint32_t)k * (uint32_t)(ldw * 2) + (uint32_t)(col0 + c * 8) * 2 : kOutOfRange;
            }
        }
        auto issue_one = [&](auto I, int i, int kstep, bool live) {
            const bool is_a = i < A_ITERS;
            const bool second = kstep >= nk1;
            const int ks = second ? kstep - nk1 : kstep;
            if (is_a) {
                const rsrc_t r = make_rsrc(second ? abase[1] : abase[0], live ? a_bytes : 0u);
                const uint32_t vo = ks * BK + lane_k < Kdim ? off[i] : kOutOfRange;
                lds_buf16<0>(r, a_base(I) + (i * NW + wave) * 1024, vo, ks * BK * 2);
            } else {
                const int left = Kdim - ks * BK < BK ? Kdim - ks * BK : BK;
                const rsrc_t r = make_rsrc((second ? wbase[1] : wbase[0]) + (size_t)ks * BK * ldw * 2,
                                           live ? (uint32_t)left * (uint32_t)(ldw * 2) : 0u);
                lds_buf16<kNonTemporal>(r, b_base(I) + ((i - A_ITERS) * NW + wave) * 1024, off[i], 0);
            }
        };

        int lds_lane[2];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
            lds_lane[kk] = (lane & 15) * ROWB + (((kk * 4 + (lane >> 4)) ^ (lane & 7)) * 16);
        uint32_t wfrag[FN];
#pragma unroll
        for (int f = 0; f < FN; ++f) wfrag[f] = frag_offset<BN>(lane, wn * (FN * 16) + f * 16);

        const int nf = __builtin_amdgcn_readfirstlane(
            nvalid > wm * 16 ? min(FM, (nvalid - wm * 16 + 31) / 32) : 0);

        // the previous tile's reads of both stages must be complete before new loads land
        wait_lgkm0();
        block_barrier();
#pragma unroll
        for (int i = 0; i < LPS; ++i) issue_one(ic<0>{}, i, 0, true);
        {
            const bool l1 = __builtin_amdgcn_readfirstlane(nk > 1 ? 1 : 0) != 0;
#pragma unroll
            for (int i = A_ITERS; i < LPS; ++i) issue_one(ic<1>{}, i, 1, l1);
        }

        auto tile = [&](auto NFc) {
            constexpr int NF = decltype(NFc)::value;
            floatx4 acc[NF > 0 ? NF : 1][FN];
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int f = 0; f < FN; ++f) acc[i][f] = floatx4{0.f, 0.f, 0.f, 0.f};

            auto compute = [&](auto I, int k, bool liveA, bool liveB) {
                const char* ab = a_base(I);
                const uint32_t bb = lds_addr(b_base(I));
                constexpr auto nextbuf = ic<1 - decltype(I)::value>{};
                uint32_t ad[FN];
#pragma unroll
                for (int f = 0; f < FN; ++f) ad[f] = bb + wfrag[f];
                bf16x8 bfr[2][FN];
                if constexpr (LOOK) {
                    read_frags<BN, 0>(bfr[0], ad);
                    read_frags<BN, 1>(bfr[1], ad);
                    block_barrier();                     // every wave holds this step's weight fragments
                }
                auto issue_slot = [&](int q) {
                    if (q < A_ITERS) issue_one(nextbuf, q, k + 1, liveA);
                    else issue_one(I, q, k + 2, liveB);
                };
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    if constexpr (!LOOK) {
                        if (kk == 0) read_frags<BN, 0>(bfr[0], ad);
                        else {
                            read_frags<BN, 1>(bfr[1], ad);
                            block_barrier();
                        }
                    }
                    bf16x8 acur;
                    if (NF > 0) acur = *reinterpret_cast<const bf16x8*>(ab + lds_lane[kk] + wm * 16 * ROWB);
#pragma unroll
                    for (int i = 0; i < NF; ++i) {
                        bf16x8 anext;
                        if (i + 1 < NF)
                            anext = *reinterpret_cast<const bf16x8*>(
                                ab + lds_lane[kk] + (wm + WMW * (i + 1)) * 16 * ROWB);
#pragma unroll
                        for (int f = 0; f < FN; ++f)
                            acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(acur, bfr[kk][f], acc[i][f], 0, 0, 0);
                        if constexpr (LOOK) {
                            const int slot = kk * NF + i;
                            if (slot < LPS) issue_slot(slot);
                        } else {
                            if (kk == 0 && i < A_ITERS) issue_slot(i);
                            if (kk == 1 && i < B_ITERS) issue_slot(A_ITERS + i);
                        }
                        if (i + 1 < NF) acur = anext;
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if constexpr (!LOOK) {
                        if (kk == 0) {
#pragma unroll
                            for (int q = NF; q < A_ITERS; ++q) issue_slot(q);
                        } else {
#pragma unroll
                            for (int q = NF; q < B_ITERS; ++q) issue_slot(A_ITERS + q);
                        }
                    }
                }
                if constexpr (LOOK) {
#pragma unroll
                    for (int q = 2 * NF; q < LPS; ++q) issue_slot(q);
                }
            };
            auto step = [&](auto I, int k) {
                wait_vmcnt<B_ITERS>();
                wait_lgkm0();
                block_barrier();
                const bool l1 = __builtin_amdgcn_readfirstlane(k + 1 < nk ? 1 : 0) != 0;
                const bool l2 = __builtin_amdgcn_readfirstlane(k + 2 < nk ? 1 : 0) != 0;
                compute(I, k, l1, l2);
            };
            for (int k = 0; k < nk; k += 2) {
                step(ic<0>{}, k);
                if (k + 1 < nk) step(ic<1>{}, k + 1);
            }
            wait_vmcnt<0>();                             // the last step's loads read nothing but count

            // epilogue: PF fragments at a time through a private LDS region, out in 16-byte chunks
            constexpr int OCOLS = FN * 16, OCH = OCOLS / 8, OPITCH = OCOLS * 2 + 16, PF = 5;
            constexpr int RSZ = PF * 16 * OPITCH, RPI = 64 / OCH;
            static_assert(2 * RSZ <= BK * BN * 2 && 2 * RSZ <= BM * ROWB, "two regions per stage buffer");
            wait_lgkm0();
            block_barrier();
            char* region = (wave < 2 ? reinterpret_cast<char*>(sa0) : wave < 4 ? reinterpret_cast<char*>(sb0)
                            : wave < 6 ? reinterpret_cast<char*>(sa1) : reinterpret_cast<char*>(sb1)) + (wave & 1) * RSZ;
            const int colbase = col0 + wn * OCOLS;
            char* out_bytes = reinterpret_cast<char*>(Out);
#pragma unroll
            for (int p0 = 0; p0 < NF; p0 += PF) {
#pragma unroll
                for (int ii = 0; ii < PF; ++ii) {
                    const int i = p0 + ii;
                    if (i < NF) {
#pragma unroll
                        for (int f = 0; f < FN; ++f)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                *reinterpret_cast<uint16_t*>(region + (ii * 16 + (lane >> 4) * 4 + e) * OPITCH +
                                                             (f * 16 + (lane & 15)) * 2) =
                                    (uint16_t)f32_to_bf16_bits(acc[i][f][e]);
                    }
                }
#pragma unroll
                for (int q = 0; q < PF * 16 / RPI; ++q) {
                    const int lrow = q * RPI + lane / OCH, ch = lane % OCH;
                    const int i = p0 + lrow / 16;
                    const int trow = (wm + WMW * i) * 16 + lrow % 16;
                    const int col = colbase + ch * 8;
                    if (i < NF && trow < nvalid && col < N)
                        *reinterpret_cast<uint4*>(out_bytes + ((size_t)(row0 + trow) * N + col) * 2) =
                            *reinterpret_cast<const uint4*>(region + lrow * OPITCH + ch * 16);
                }
            }
        };
        static_assert(FM <= 10, "one case per fragment count");
        switch (nf) {
            case 0: tile(ic<0>{}); break;
            case 1: tile(ic<1>{}); break;
            case 2: tile(ic<2>{}); break;
            case 3: tile(ic<3>{}); break;
            case 4: tile(ic<4>{}); break;
            case 5: tile(ic<5>{}); break;
            case 6: tile(ic<6>{}); break;
            case 7: tile(ic<7>{}); break;
            case 8: tile(ic<8>{}); break;
            case 9: if constexpr (9 <= FM) tile(ic<9>{}); break;
            case 10: if constexpr (10 <= FM) tile(ic<10>{}); break;
            default: break;
        }
    }
}

// ---- few rows: register-staged tiles of BM rows by 128 columns, as ffn_bf16.hip's
template <int BM, int WMW, int WNW>
__global__ __launch_bounds__(64 * WMW * WNW) void dgrad_small_kernel(FfnArgs p) {
    constexpr int NT = 64 * WMW * WNW, TW = 128;
    constexpr int FM = BM / 16 / WMW, WN = TW / WNW, FN = WN / 16;
    constexpr int A_IT = (BM * 8 + NT - 1) / NT, B_IT = BK * TW / 8 / NT;
    static_assert(FM >= 1 && FN >= 1 && B_IT * NT == BK * TW / 8, "tile shape");

    __shared__ uint4 sA[BM * 8];
    __shared__ uint4 sB[BK * TW / 8];
    __shared__ int s_row[BM];
    __shared__ int s_pre[kMaxExperts + 1];
    __shared__ int s_tmp[NT / kWave];

    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int wm = wave / WNW, wn = wave % WNW;
    const int Kdim = p.Kdim, N = p.N, ldw = p.ldw;
    build_tile_prefix<NT, BM>(p, s_pre, s_tmp);
    const int n_tiles_n = (N + TW - 1) / TW;
    const int total = n_tiles_n * s_pre[p.E_loc];
    const int G = gridDim.x, v = xcd_block_order();
    uint16_t* __restrict__ Out = static_cast<uint16_t*>(p.out);
    uint32_t wfrag[FN];
#pragma unroll
    for (int f = 0; f < FN; ++f) wfrag[f] = frag_offset<TW>(lane, wn * WN + f * 16);

    for (int rnd = 0;; ++rnd) {
        const int tau = round_tile(rnd, v, blockIdx.x, G, total);
        if (tau < 0) break;
        const TileCoord tc = decode_tile<BM>(tau, n_tiles_n, s_pre, p);
        const int row0 = tc.row0, nvalid = tc.nvalid, col0 = tc.nt * TW;
        __syncthreads();                                 // the previous tile's reads are done
        for (int r = tid; r < BM; r += NT) s_row[r] = r < nvalid ? dy_row(p, row0 + r) : -1;
        __syncthreads();

        floatx4 acc[FM][FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int f = 0; f < FN; ++f) acc[i][f] = floatx4{0.f, 0.f, 0.f, 0.f};

        for (int q = 0; q < 2; ++q) {
            const uint16_t* A = static_cast<const uint16_t*>(q == 0 ? p.a : p.a2);
            if (A == nullptr) break;
            const uint16_t* W = static_cast<const uint16_t*>(q == 0 ? p.w0 : p.w1) + (size_t)tc.j * Kdim * ldw;
            uint4 ra[A_IT], rb[B_IT];
            auto load_step = [&](int k0) {
#pragma unroll
                for (int i = 0; i < A_IT; ++i) {
                    const int e = tid + i * NT, r = e >> 3, c = e & 7;
                    const int row = e < BM * 8 ? s_row[r] : -1;
                    ra[i] = row >= 0 && k0 + c * 8 < Kdim
                                ? *reinterpret_cast<const uint4*>(A + (size_t)row * Kdim + k0 + c * 8)
                                : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < B_IT; ++i) {
                    const int e = tid + i * NT, k = e / (TW / 8), c = e % (TW / 8);
                    rb[i] = k0 + k < Kdim && col0 + c * 8 < N ? load_stream16(W + (size_t)(k0 + k) * ldw + col0 + c * 8)
                                                              : make_uint4(0, 0, 0, 0);
                }
            };
            load_step(0);
            for (int k0 = 0; k0 < Kdim; k0 += BK) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < A_IT; ++i) {
                    const int e = tid + i * NT, r = e >> 3, c = e & 7;
                    if (e < BM * 8) sA[r * 8 + (c ^ (r & 7))] = ra[i];
                }
#pragma unroll
                for (int i = 0; i < B_IT; ++i) {
                    const int e = tid + i * NT, k = e / (TW / 8), c = e % (TW / 8);
                    sB[k * (TW / 8) + (c ^ swz_row<TW>(k))] = rb[i];
                }
                __syncthreads();
                if (k0 + BK < Kdim) load_step(k0 + BK);
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const int chunk = kk * 4 + (lane >> 4);
                    bf16x8 bfr[FN];
#pragma unroll
                    for (int f = 0; f < FN; ++f) bfr[f] = read_frag<TW>(reinterpret_cast<const char*>(sB), wfrag[f], kk);
#pragma unroll
                    for (int i = 0; i < FM; ++i) {
                        const int mrow = (wm + WMW * i) * 16;
                        if (mrow < nvalid) {
                            const int r = mrow + (lane & 15);
                            const bf16x8 afr = __builtin_bit_cast(bf16x8, sA[r * 8 + (chunk ^ (r & 7))]);
#pragma unroll
                            for (int f = 0; f < FN; ++f)
                                acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(afr, bfr[f], acc[i][f], 0, 0, 0);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                const int col = col0 + wn * WN + f * 16 + (lane & 15);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = (wm + WMW * i) * 16 + (lane >> 4) * 4 + e;
                    if (r < nvalid && col < N)
                        Out[(size_t)(row0 + r) * N + col] = (uint16_t)f32_to_bf16_bits(acc[i][f][e]);
                }
            }
    }
}

template <int BM>
hipError_t launch_wide(const FfnArgs& a, hipStream_t stream) {
    static int per_cu = 0;
    return launch_persistent(dgrad_wide_kernel<BM>, 512, a, stream, &per_cu);
}
template <int BM, int WMW, int WNW>
hipError_t launch_small(const FfnArgs& a, hipStream_t stream) {
    static int per_cu = 0;
    return launch_persistent(dgrad_small_kernel<BM, WMW, WNW>, 64 * WMW * WNW, a, stream, &per_cu);
}

}  // namespace

hipError_t launch_dgrad_bf16(const FfnArgs& a, hipStream_t stream) {
    // the wide tiles address a tile's rows (gathered: all of dy) and a step's weight rows
    // with 32-bit offsets that stay below kOutOfRange, the k-step's included
    const unsigned long long reach = a.src_of != nullptr ? (unsigned long long)a.src_rows : 320;
    const bool wide_ok = (reach * a.Kdim + a.Kdim + 64) * 2 < (1ull << 31) &&
                         (unsigned long long)BK * a.ldw * 2 < (1ull << 31) && (a.src_of == nullptr || a.src_rows > 0);
    if (wide_ok && a.rows_hint >= 192) return launch_wide<320>(a, stream);
    if (wide_ok && a.rows_hint >= 64) return launch_wide<256>(a, stream);
    if (a.rows_hint < 24) return launch_small<16, 1, 2>(a, stream);
    return launch_small<128, 2, 2>(a, stream);
}

}  // namespace moeep
