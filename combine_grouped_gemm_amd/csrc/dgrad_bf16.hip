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

#define INLINE __attribute__((always_inline))

// row of dy that expert row r reads (-1: none)
__device__ __forceinline__ int dy_row(const FfnArgs& p, int r) {
    if (p.src_of == nullptr) return r;
    const int s = p.src_of[r];
    if (s < 0) return -1;
    const int t = token_of(s, p.per_div);
    return t < p.src_rows ? t : -1;
}

// ---- 8 waves 2 (rows) x 4 (columns), tiles of up to 320 rows by 256 columns.  A ring of
// 64-row stages of the contraction; how deep is a matter of the tile's rows, for the LDS is
// shared out in blocks of 64 rows of dy (8 KB), ten of them, and two stages of weights:
//   193 to 320 rows  two row stages of five blocks, rows issued one step ahead
//   129 to 192       three of three, rows two steps ahead
//   up to 128        three of two, and the last four blocks are a third weight stage
// Weights are issued as many steps ahead as they have stages (of tiles of more than 192 rows
// the next ones only half-way through the step): up to 192 rows a wave holds both halves'
// fragments of a step in registers, so that the stage is free before the step's matrix
// instructions.
// What bounds it, 32 experts of 7168 x 2048 (256 tiles, one a CU): up to 128 rows each the
// stream of weights (16 rows 146 us, 128 rows 155: 6.4 and 6.1 TB/s; over one set of operands 141
// and 151, with two stages of each 150 and 160); from 192 rows on the matrix instructions beside
// it (256 rows 221 us, 1.09 PFLOP/s; 640 rows 476 us, 1.26); of ragged experts the rounds that
// tiles of unlike cost do not fill (a rank with 26 to 1131 rows an expert, 336 to 400 tiles: 275
// us).  A pair at 2880 x 2880, 128 experts of 128 rows on average: 865 us, with two stages 980.
constexpr int kBM = 320;

// A tile's plan: MODE 0, 1, 2 as above with the row fragments NF of a wave
template <int MODE>
struct Plan {
    static constexpr int A_ITERS = MODE == 0 ? 2 : MODE == 1 ? 3 : 5;    // 64-row blocks of a stage
    static constexpr int AST = MODE == 2 ? 2 : 3, BST = MODE == 0 ? 3 : 2;
    static constexpr int DA = AST - 1, DB = BST;                         // steps ahead that are issued
    static constexpr int UNROLL = MODE == 0 ? 3 : MODE == 1 ? 6 : 2;
    static constexpr bool LOOK = MODE < 2;
};

__global__ __launch_bounds__(512, 1) void dgrad_wide_kernel(FfnArgs p) {
    constexpr int WMW = 2, WNW = 4, NT = 512, NW = 8;
    constexpr int A_MAX = kBM / 64;                  // row loads of a wave per stage: 8 rows each
    constexpr int B_ITERS = BK * BN * 2 / 1024 / NW; // weight loads: 1 KiB is two rows of 256 columns
    constexpr int FN = BN / WNW / 16;
    constexpr int BLK = 64 * ROWB;                   // a block of 64 rows
    static_assert(B_ITERS == 4 && FN == 4 && BLK == 8192, "tile shape");

    // each block and stage an object of its own: the compiler sees that reads of one do not
    // depend on the loads in flight into the others
    __shared__ uint4 s_b0[BK * BN / 8], s_b1[BK * BN / 8];
    __shared__ uint4 s_r0[BLK / 16], s_r1[BLK / 16], s_r2[BLK / 16], s_r3[BLK / 16], s_r4[BLK / 16], s_r5[BLK / 16];
    __shared__ uint4 s_r6[4 * BLK / 16];             // blocks 6 to 9, or the third weight stage
    __shared__ int s_pre[kMaxExperts + 1];
    __shared__ uint16_t s_ord[kMaxExperts];
    static_assert(sizeof(s_b0) >= 2 * kMaxExperts * sizeof(int), "row counts and blocks' loads fit in the first weight stage");
    static_assert(sizeof(s_r6) == sizeof(s_b0), "a weight stage");
    __shared__ int s_tmp[NT / kWave];

    auto block = [&](int b) INLINE -> char* {
        uint4* q = b == 0 ? s_r0 : b == 1 ? s_r1 : b == 2 ? s_r2 : b == 3 ? s_r3 : b == 4 ? s_r4 : b == 5 ? s_r5
                   : s_r6 + (b - 6) * (BLK / 16);
        return reinterpret_cast<char*>(q);
    };

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / WNW, wn = wave % WNW;
    const int Kdim = p.Kdim, N = p.N, ldw = p.ldw;
    const int nk1 = (Kdim + BK - 1) / BK, nk = p.a2 != nullptr ? 2 * nk1 : nk1;
    const int lane_k = swz(lane / 8, lane % 8) * 8;

    build_tile_prefix_sorted<NT, kBM, true>(p, s_pre, s_ord, reinterpret_cast<int*>(s_b0), s_tmp);
    const int n_tiles_n = (N + BN - 1) / BN;
    const int total = __builtin_amdgcn_readfirstlane(n_tiles_n * s_pre[p.E_loc]);
    const int G = gridDim.x;
    const int v = total <= G ? xcd_chunk_order() : xcd_block_order();

    const int full = total / G;
    int last = round_tile_back(full, v, G, total);
    if (full > 0 && full <= kLookBack && total > full * G && G <= kMaxExperts)
        last = last_round_tile<NT, kBM>(full, v, G, total, n_tiles_n, p.E_loc, s_pre, s_ord, reinterpret_cast<int*>(s_b0), s_tmp);
    for (int rnd = 0; rnd <= full; ++rnd) {
        const int tau = rnd < full ? round_tile_back(rnd, v, G, total) : last;
        if (tau < 0) break;
        const TileCoord tc = decode_tile<kBM>(tau, n_tiles_n, s_pre, p, s_ord);
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
        uint32_t aoff[A_MAX], boff[B_ITERS];
#pragma unroll
        for (int i = 0; i < A_MAX; ++i) {
            const int r = (i * NW + wave) * 8 + lane / 8;
            int q = -1;
            if (r < nvalid) q = p.src_of != nullptr ? dy_row(p, row0 + r) : r;
            aoff[i] = q >= 0 ? (uint32_t)q * (uint32_t)(Kdim * 2) + (uint32_t)swz(r, lane % 8) * 16 : kOutOfRange;
        }
#pragma unroll
        for (int i = 0; i < B_ITERS; ++i) {
            const int k = (i * NW + wave) * 2 + lane / 32;
            const int c = (lane % 32) ^ swz_row<BN>(k);
            boff[i] = col0 + c * 8 < N ? (uint32_t)k * (uint32_t)(ldw * 2) + (uint32_t)(col0 + c * 8) * 2 : kOutOfRange;
        }

        int lds_lane[2];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
            lds_lane[kk] = (wm * 16 + (lane & 15)) * ROWB + (((kk * 4 + (lane >> 4)) ^ (lane & 7)) * 16);
        uint32_t wfrag[FN];
#pragma unroll
        for (int f = 0; f < FN; ++f) wfrag[f] = frag_offset<BN>(lane, wn * (FN * 16) + f * 16);

        // the previous tile's reads of every stage must be complete before new loads land
        wait_lgkm0();
        block_barrier();

        auto tile = [&](auto NFc, auto MODEc) INLINE {
            constexpr int NF = decltype(NFc)::value, MODE = decltype(MODEc)::value;
            using P = Plan<MODE>;
            constexpr int A_ITERS = P::A_ITERS, LPS = A_ITERS + B_ITERS;
            // step k's stages, by its index in the unrolled loop: row fragment i's, and the weights'
            auto a_block = [&](auto I, int b) INLINE { return block(decltype(I)::value % P::AST * A_ITERS + b); };
            auto b_base = [&](auto I) INLINE -> char* {
                constexpr int s = decltype(I)::value % P::BST;
                return reinterpret_cast<char*>(s == 0 ? s_b0 : s == 1 ? s_b1 : s_r6);
            };
            auto issue_a = [&](auto I, int i, int kstep, bool live) INLINE {
                const bool second = kstep >= nk1;
                const int ks = second ? kstep - nk1 : kstep;
                const rsrc_t r = make_rsrc(second ? abase[1] : abase[0], live ? a_bytes : 0u);
                const uint32_t vo = ks * BK + lane_k < Kdim ? aoff[i] : kOutOfRange;
                lds_buf16<0>(r, a_block(I, i) + wave * 1024, vo, ks * BK * 2);
            };
            auto issue_b = [&](auto I, int i, int kstep, bool live) INLINE {
                const bool second = kstep >= nk1;
                const int ks = second ? kstep - nk1 : kstep;
                const int left = Kdim - ks * BK < BK ? Kdim - ks * BK : BK;
                const rsrc_t r = make_rsrc((second ? wbase[1] : wbase[0]) + (size_t)ks * BK * ldw * 2,
                                           live ? (uint32_t)left * (uint32_t)(ldw * 2) : 0u);
                lds_buf16<kNonTemporal>(r, b_base(I) + (i * NW + wave) * 1024, boff[i], 0);
            };
            auto live_step = [&](int k) INLINE { return __builtin_amdgcn_readfirstlane(k < nk ? 1 : 0) != 0; };
            auto first_step = [&](auto I) INLINE {
                constexpr int k = decltype(I)::value;
                const bool live = live_step(k);
                if constexpr (k < P::DA) {
#pragma unroll
                    for (int i = 0; i < A_ITERS; ++i) issue_a(I, i, k, live);
                }
                if constexpr (k < P::DB) {
#pragma unroll
                    for (int i = 0; i < B_ITERS; ++i) issue_b(I, i, k, live);
                }
            };
            first_step(ic<0>{});
            first_step(ic<1>{});
            first_step(ic<2>{});

            // the weights are the matrix instructions' row operand: a lane's four results are
            // neighbouring columns of row l % 16
            floatx4 acc[NF > 0 ? NF : 1][FN];
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int f = 0; f < FN; ++f) acc[i][f] = floatx4{0.f, 0.f, 0.f, 0.f};

            auto step = [&](auto I, int k) INLINE {
                // rows and weights of step k were issued DA and DB steps ago, rows first
                wait_vmcnt<(P::DA - 1) * LPS + (P::DB > P::DA ? B_ITERS : 0)>();
                wait_lgkm0();
                block_barrier();
                const bool liveA = live_step(k + P::DA), liveB = live_step(k + P::DB);
                auto issue_slot = [&](int q) INLINE {
                    if (q < A_ITERS) issue_a(ic<decltype(I)::value + P::DA>{}, q, k + P::DA, liveA);
                    else issue_b(I, q - A_ITERS, k + P::DB, liveB);
                };
                auto row_frag = [&](int kk, int i) INLINE {
                    return *reinterpret_cast<const bf16x8*>(a_block(I, i / 2) + (i & 1) * (WMW * 16 * ROWB) + lds_lane[kk]);
                };
                const uint32_t bb = lds_addr(b_base(I));
                uint32_t ad[FN];
#pragma unroll
                for (int f = 0; f < FN; ++f) ad[f] = bb + wfrag[f];
                bf16x8 bfr[2][FN];
                if constexpr (P::LOOK) {
                    read_frags<BN, 0>(bfr[0], ad);
                    read_frags<BN, 1>(bfr[1], ad);
                    block_barrier();                     // every wave holds this step's weight fragments
                }
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    if constexpr (!P::LOOK) {
                        if (kk == 0) read_frags<BN, 0>(bfr[0], ad);
                        else {
                            read_frags<BN, 1>(bfr[1], ad);
                            block_barrier();
                        }
                    }
                    bf16x8 acur;
                    if (NF > 0) acur = row_frag(kk, 0);
#pragma unroll
                    for (int i = 0; i < NF; ++i) {
                        bf16x8 anext;
                        if (i + 1 < NF) anext = row_frag(kk, i + 1);
#pragma unroll
                        for (int f = 0; f < FN; ++f)
                            acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bfr[kk][f], acur, acc[i][f], 0, 0, 0);
                        if constexpr (P::LOOK) {
                            const int slot = kk * NF + i;
                            if (slot < LPS) issue_slot(slot);
                        } else {
                            if (kk == 0 && i < A_ITERS) issue_slot(i);
                            if (kk == 1 && i < B_ITERS) issue_slot(A_ITERS + i);
                        }
                        if (i + 1 < NF) acur = anext;
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                if constexpr (P::LOOK) {
#pragma unroll
                    for (int q = 2 * NF; q < LPS; ++q) issue_slot(q);
                } else {
                    static_assert(NF >= A_ITERS && NF >= B_ITERS, "a slot for every load");
                }
            };
            for (int k = 0; k < nk; k += P::UNROLL) {
                step(ic<0>{}, k);
                if (k + 1 < nk) step(ic<1>{}, k + 1);
                if constexpr (P::UNROLL > 2) {
                    if (k + 2 < nk) step(ic<2>{}, k + 2);
                }
                if constexpr (P::UNROLL > 3) {
                    if (k + 3 < nk) step(ic<3>{}, k + 3);
                    if (k + 4 < nk) step(ic<4>{}, k + 4);
                    if (k + 5 < nk) step(ic<5>{}, k + 5);
                }
            }
            wait_vmcnt<0>();                             // the last steps' loads read nothing but count

            // out: lanes exchange values so that each holds 16 bytes of a row, 8 lanes a
            // whole line of the wave's 64 columns
            int ln = lane;
            asm volatile("" : "+v"(ln));                 // keeps what depends on it out of the k-loop's registers
            uint16_t* Out = static_cast<uint16_t*>(p.out) + (size_t)row0 * N;
            const int col = col0 + wn * (FN * 16) + unit_col(ln);
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                uint4 u[2];
                units_of(acc[i], u);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = (wm + WMW * i) * 16 + h * 8 + (ln & 7);
                    if (r < nvalid && col < N) *reinterpret_cast<uint4*>(Out + (size_t)r * N + col) = u[h];
                }
            }
        };
        const int nf = __builtin_amdgcn_readfirstlane(nvalid > wm * 16 ? (nvalid - wm * 16 + 31) / 32 : 0);
        if (nvalid <= 128) {
            switch (nf) {
                case 0: tile(ic<0>{}, ic<0>{}); break;
                case 1: tile(ic<1>{}, ic<0>{}); break;
                case 2: tile(ic<2>{}, ic<0>{}); break;
                case 3: tile(ic<3>{}, ic<0>{}); break;
                default: tile(ic<4>{}, ic<0>{}); break;
            }
        } else if (nvalid <= 192) {
            switch (nf) {
                case 4: tile(ic<4>{}, ic<1>{}); break;
                case 5: tile(ic<5>{}, ic<1>{}); break;
                default: tile(ic<6>{}, ic<1>{}); break;
            }
        } else {
            switch (nf) {
                case 6: tile(ic<6>{}, ic<2>{}); break;
                case 7: tile(ic<7>{}, ic<2>{}); break;
                case 8: tile(ic<8>{}, ic<2>{}); break;
                case 9: tile(ic<9>{}, ic<2>{}); break;
                default: tile(ic<10>{}, ic<2>{}); break;
            }
        }
    }
}

// ---- register-staged tiles of BM rows by 128 columns, as ffn_bf16.hip's, with 64-bit addresses
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
    const int G = gridDim.x, v = total <= G ? xcd_chunk_order() : xcd_block_order();
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

hipError_t launch_wide(const FfnArgs& a, hipStream_t stream) {
    static int per_cu = 0;
    return launch_persistent(dgrad_wide_kernel, 512, a, stream, &per_cu);
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
    if (!wide_ok) return launch_small<128, 2, 2>(a, stream);
    // a few rows and a short contraction: several small blocks a CU hide the rings' filling and
    // the epilogue (64 experts of 2 rows, 512 x 512: 12.8 us, wide 17.3; at 1024 x 1024 they meet,
    // 32 experts of 4 rows 21.6 and 20.2; 32 of 8 rows, 7168 x 2048: 266 and 144)
    if (a.rows_hint < 24 && a.Kdim <= 1024) return launch_small<16, 1, 2>(a, stream);
    return launch_wide(a, stream);
}

}  // namespace moeep
