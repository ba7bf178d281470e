// Weight gradients of the grouped products in bf16: dw_j = base_j + sum over expert j's
// rows r of dy[r]^T x[r], for one or two dy that share x; fp32 accumulation on MFMA.
//
// Both operands are contracted over their rows, so a k-step is 64 rows of the tile's
// columns of each, as they are in memory, and every fragment is a transposing LDS read
// (gemm_cols.hpp).  The matrix cores get x as their row operand: a lane's four results
// are then four neighbouring columns of one dw row, stored as one piece.
//
// What bounds it is writing dw: with a few hundred rows an expert a 256 x 256 tile has 4 to
// 8 steps and 256 KB of fp32 to write.  So the steps of all of a block's tiles run as one
// sequence: the first step of the next tile is loaded under the last one of this tile,
// and the tile's stores drain under the next tile's steps.
//
// The row of a gathered operand (src_of) is looked up once per piece of work (a tile, or
// 1024 rows of one): the piece's rows are listed in LDS during the piece before, so that a
// load's address is one LDS read away.  Rows past the expert's last one, and rows that
// src_of names nowhere, get an offset outside the operand's extent, read nothing and land
// zeros in both operands.
//
// A checkpoint x comes through registers: 16 codes a load, issued a step ahead as the
// direct loads are, turned into the bf16 values they stand for (exact) after the step's
// matrix instructions and written to the stage that the next step reads.
#include "ckpt_common.hpp"
#include "gemm_cols.hpp"

namespace moeep {
namespace {

using namespace cols;

constexpr int kPieceRows = 1024;             // rows listed at a time
#define INLINE __attribute__((always_inline))

// what a lane of a 64-bit gathered load reads where there is no row
__device__ uint4 g_zeros;

// TN, TM: tile of dw (out x in).  8 waves, 2 (out) x 4 (in).  FAR: a gathered operand of
// 2 GiB or more, which a buffer resource's 32-bit offsets do not reach: 64-bit addresses.
template <int TN, int TM, bool CKPT, bool FAR>
__global__ __launch_bounds__(512, 1) void wgrad_kernel(WgradArgs p, int tiles_n, int tiles_m, int tiles) {
    constexpr int NT = 512, NW = 8;
    constexpr int FN = TN / 2 / 16, FM = TM / 4 / 16;        // fragments of a wave
    constexpr int Y_ITERS = BK * TN * 2 / 1024 / NW;         // direct loads of a wave per step
    constexpr int X_ITERS = BK * TM * 2 / 1024 / NW;
    constexpr int C_ITERS = BK * TM / 1024 / NW;             // checkpoint: 16-code loads of a lane
    constexpr int YR = 512 / TN, XR = 512 / TM;              // rows of a direct load
    constexpr int CR = 1024 / TM;                            // rows of a wave's code load
    static_assert(Y_ITERS >= 1 && X_ITERS >= 1 && C_ITERS >= 1, "tile shape");

    __shared__ uint4 sy0[BK * TN / 8];
    __shared__ uint4 sx0[BK * TM / 8];
    __shared__ uint4 sy1[BK * TN / 8];
    __shared__ uint4 sx1[BK * TM / 8];
    __shared__ int s_tok[2][kPieceRows];

    auto y_base = [&](auto I) -> char* {
        if constexpr (decltype(I)::value == 0) return reinterpret_cast<char*>(sy0);
        else return reinterpret_cast<char*>(sy1);
    };
    auto x_base = [&](auto I) -> char* {
        if constexpr (decltype(I)::value == 0) return reinterpret_cast<char*>(sx0);
        else return reinterpret_cast<char*>(sx1);
    };

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wn = wave / 4, wm = wave % 4;
    const int N = p.N, M = p.M;
    const int nb = (M + kCkptBlock - 1) / kCkptBlock;
    const bool gathers = p.src_of != nullptr;

    // a piece of work: rows [row0, row0 + rows) of a tile's expert
    struct Piece {
        int tile;
        int j, q, n0, m0, row0, rows, end;      // end: the expert's last row, exclusive
    };
    auto open_tile = [&](int tau, Piece& w) INLINE {
        w.tile = tau;
        if (tau >= tiles) return;
        // the tiles of one expert's one dw, columns (in) slowest: tiles that run together share both operands
        unsigned rest = (unsigned)tau;
        w.n0 = (int)(rest % (unsigned)tiles_n) * TN;
        rest /= (unsigned)tiles_n;
        const unsigned pairs = p.dy[1] != nullptr ? 2 : 1;
        w.q = (int)(rest % pairs);
        rest /= pairs;
        w.m0 = (int)(rest % (unsigned)tiles_m) * TM;
        w.j = (int)(rest / (unsigned)tiles_m);
        w.row0 = clampi(p.offsets[w.j], 0, p.cap);
        w.end = clampi(p.offsets[w.j + 1], w.row0, p.cap);
        w.n0 = __builtin_amdgcn_readfirstlane(w.n0);
        w.q = __builtin_amdgcn_readfirstlane(w.q);
        w.m0 = __builtin_amdgcn_readfirstlane(w.m0);
        w.j = __builtin_amdgcn_readfirstlane(w.j);
        w.row0 = __builtin_amdgcn_readfirstlane(w.row0);
        w.end = __builtin_amdgcn_readfirstlane(w.end);
        w.rows = min(w.end - w.row0, kPieceRows);
    };
    const int G = gridDim.x;
    auto after = [&](const Piece& w) INLINE {
        Piece n = w;
        if (w.row0 + w.rows < w.end) {
            n.row0 = w.row0 + w.rows;
            n.rows = min(w.end - n.row0, kPieceRows);
        } else {
            open_tile(w.tile < tiles - G ? w.tile + G : tiles, n);
        }
        return n;
    };
    // the slots of a piece's rows, and the list of the rows that a gathered operand reads for them
    constexpr int LIST = kPieceRows / NT;
    int listed[LIST];
    auto load_list = [&](const Piece& w) INLINE {
        if (!gathers || w.tile >= tiles) return;
#pragma unroll
        for (int i = 0; i < LIST; ++i) {
            const int r = i * NT + tid;
            listed[i] = r < w.rows ? p.src_of[w.row0 + r] : -1;
        }
    };
    auto store_list = [&](const Piece& w, int* tok) INLINE {
        if (!gathers || w.tile >= tiles) return;
#pragma unroll
        for (int i = 0; i < LIST; ++i) {
            const int t = listed[i] < 0 ? -1 : token_of(listed[i], p.per_div);
            tok[i * NT + tid] = t < p.src_rows ? t : -1;
        }
    };

    // direct load i of an operand's step: `i0` first row of the step within the piece
    auto row_at = [&](const Piece& w, const int* tok, bool gathered, int i) INLINE -> int {
        if (i >= w.rows) return -1;
        return gathered ? tok[i] : w.row0 + i;
    };
    auto issue_y = [&](auto I, const Piece& w, const int* tok, int i0, int i) INLINE {
        const int blk = i * NW + wave, k = blk * YR + lane / (64 / YR);
        const int c = (lane % (64 / YR)) ^ swz_row<TN>(k);
        const int col = w.n0 + c * 8;
        const int r = row_at(w, tok, p.gather_dy, i0 + k);
        // gathered rows lie anywhere, others within the expert's
        const char* base = static_cast<const char*>(w.q == 0 ? p.dy[0] : p.dy[1]) +
                           (p.gather_dy ? (size_t)0 : (size_t)w.row0 * N * 2);
        const int rel = p.gather_dy ? r : i0 + k;
        const uint32_t bytes = (uint32_t)(p.gather_dy ? p.src_rows : w.rows) * (uint32_t)(N * 2);
        const bool here = r >= 0 && col < N;
        char* dst = y_base(I) + blk * 1024;
        if constexpr (FAR)
            lds_dma16<0>(here ? base + (size_t)rel * N * 2 + col * 2 : reinterpret_cast<const char*>(&g_zeros), dst);
        else
            lds_buf16<0>(make_rsrc(base, bytes), dst, here ? (uint32_t)rel * (uint32_t)(N * 2) + (uint32_t)col * 2 : kOutOfRange, 0);
    };
    auto issue_x = [&](auto I, const Piece& w, const int* tok, int i0, int i) INLINE {
        const int blk = i * NW + wave, k = blk * XR + lane / (64 / XR);
        const int c = (lane % (64 / XR)) ^ swz_row<TM>(k);
        const int col = w.m0 + c * 8;
        const int r = row_at(w, tok, p.gather_x, i0 + k);
        const char* base = static_cast<const char*>(p.x) + (p.gather_x ? (size_t)0 : (size_t)w.row0 * M * 2);
        const int rel = p.gather_x ? r : i0 + k;
        const uint32_t bytes = (uint32_t)(p.gather_x ? p.src_rows : w.rows) * (uint32_t)(M * 2);
        const bool here = r >= 0 && col < M;
        char* dst = x_base(I) + blk * 1024;
        if constexpr (FAR)
            lds_dma16<0>(here ? base + (size_t)rel * M * 2 + col * 2 : reinterpret_cast<const char*>(&g_zeros), dst);
        else
            lds_buf16<0>(make_rsrc(base, bytes), dst, here ? (uint32_t)rel * (uint32_t)(M * 2) + (uint32_t)col * 2 : kOutOfRange, 0);
    };
    // 16 codes of a row and their scale (zeros where there is no row)
    uint4 code[C_ITERS];
    float cscale[C_ITERS];
    auto load_codes = [&](const Piece& w, const int* tok, int i0) INLINE {
#pragma unroll
        for (int i = 0; i < C_ITERS; ++i) {
            const int k = (i * NW + wave) * CR + lane / (TM / 16);
            const int col = w.m0 + (lane % (TM / 16)) * 16;
            const int r = row_at(w, tok, p.gather_x, i0 + k);
            code[i] = make_uint4(0, 0, 0, 0);
            cscale[i] = 0.0f;
            if (r >= 0 && col < M) {
                const int8_t* row = static_cast<const int8_t*>(p.x) + (size_t)r * M + col;
                const uint2 lo = *reinterpret_cast<const uint2*>(row);
                uint2 hi = make_uint2(0, 0);
                if (col + 8 < M) hi = *reinterpret_cast<const uint2*>(row + 8);
                code[i] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                cscale[i] = p.x_scales[(size_t)r * nb + col / kCkptBlock];
            }
        }
    };
    auto store_codes = [&](auto I) INLINE {
#pragma unroll
        for (int i = 0; i < C_ITERS; ++i) {
            const int k = (i * NW + wave) * CR + lane / (TM / 16), c = (lane % (TM / 16)) * 2;
            const float s = cscale[i];
            const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[e * 2] = pack_bf16x2(code_value<0>(w[e]) * s, code_value<1>(w[e]) * s);
                o[e * 2 + 1] = pack_bf16x2(code_value<2>(w[e]) * s, code_value<3>(w[e]) * s);
            }
            // both chunks of a 32-byte pair move together under the XOR
            uint4* d = reinterpret_cast<uint4*>(x_base(I) + k * TM * 2 + (c ^ swz_row<TM>(k)) * 16);
            d[0] = make_uint4(o[0], o[1], o[2], o[3]);
            d[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    };

    uint32_t yfrag[FN], xfrag[FM];
#pragma unroll
    for (int f = 0; f < FN; ++f) yfrag[f] = frag_offset<TN>(lane, wn * (FN * 16) + f * 16);
#pragma unroll
    for (int f = 0; f < FM; ++f) xfrag[f] = frag_offset<TM>(lane, wm * (FM * 16) + f * 16);

    floatx4 acc[FN][FM];
    auto clear = [&]() INLINE {
#pragma unroll
        for (int a = 0; a < FN; ++a)
#pragma unroll
            for (int b = 0; b < FM; ++b) acc[a][b] = floatx4{0.f, 0.f, 0.f, 0.f};
    };
    clear();

    // dw of a finished tile: lane l has row n = l % 16 and columns 4 (l / 16) .. + 3 of every fragment
    auto write_tile = [&](const Piece& w) INLINE {
        const size_t mat = (size_t)w.j * N * M;
        const void* base = w.q == 0 ? p.base[0] : p.base[1];
        void* dw = w.q == 0 ? p.dw[0] : p.dw[1];
#pragma unroll
        for (int a = 0; a < FN; ++a) {
            const int n = w.n0 + wn * (FN * 16) + a * 16 + (lane & 15);
            const size_t row = mat + (size_t)n * M;
            floatx4 b[FM];
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const int m = w.m0 + wm * (FM * 16) + f * 16 + (lane >> 4) * 4;
                b[f] = floatx4{0.f, 0.f, 0.f, 0.f};
                if (base != nullptr && n < N && m < M) {
                    if (p.dw_f32) {
                        const float4 t = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + row + m);
                        b[f] = floatx4{t.x, t.y, t.z, t.w};
                    } else {
                        const uint2 t = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + row + m);
                        b[f] = floatx4{bf16_lo(t.x), bf16_hi(t.x), bf16_lo(t.y), bf16_hi(t.y)};
                    }
                }
            }
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                const int m = w.m0 + wm * (FM * 16) + f * 16 + (lane >> 4) * 4;
                if (n >= N || m >= M) continue;
                const floatx4 s = acc[a][f] + b[f];
                if (p.dw_f32)
                    *reinterpret_cast<float4*>(static_cast<float*>(dw) + row + m) = make_float4(s[0], s[1], s[2], s[3]);
                else
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dw) + row + m) =
                        make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
            }
        }
    };

    // the sequence of steps: `cur` is computed, `nxt` loaded
    Piece cur, nxt;
    open_tile(xcd_block_order(), cur);
    if (cur.tile >= tiles) return;
    int slot = 0;                                            // s_tok of cur's piece; the next one's is the other
    load_list(cur);
    store_list(cur, s_tok[0]);
    nxt = after(cur);
    load_list(nxt);
    store_list(nxt, s_tok[1]);
    __syncthreads();
    auto issue_step = [&](auto I, const Piece& w, const int* tok, int i0) INLINE {
        if constexpr (CKPT) load_codes(w, tok, i0);
#pragma unroll
        for (int i = 0; i < Y_ITERS; ++i) issue_y(I, w, tok, i0, i);
        if constexpr (!CKPT) {
#pragma unroll
            for (int i = 0; i < X_ITERS; ++i) issue_x(I, w, tok, i0, i);
        }
    };
    issue_step(ic<0>{}, cur, s_tok[0], 0);
    if constexpr (CKPT) store_codes(ic<0>{});
    int i0 = 0;                                              // first row of cur's step

    // one step; false after the last one of all
    auto step = [&](auto I) INLINE -> bool {
        constexpr auto other = ic<1 - decltype(I)::value>{};
        wait_vmcnt<0>();
        wait_lgkm0();
        block_barrier();
        // what comes next: another step of this piece, or the first of the next piece
        const bool same = __builtin_amdgcn_readfirstlane(i0 + BK < cur.rows ? 1 : 0) != 0;
        const bool more = __builtin_amdgcn_readfirstlane(same || nxt.tile < tiles ? 1 : 0) != 0;
        const bool turn = !same && more;
        Piece then = nxt;
        if (turn) {
            then = after(nxt);
            load_list(then);
        }
        if (more) {
            if (same) issue_step(other, cur, s_tok[slot], i0 + BK);
            else issue_step(other, nxt, s_tok[slot ^ 1], 0);
        }
        const char* yb = y_base(I);
        const char* xb = x_base(I);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            bf16x8 xf[FM];
#pragma unroll
            for (int f = 0; f < FM; ++f) xf[f] = read_frag<TM>(xb, xfrag[f], kk);
#pragma unroll
            for (int a = 0; a < FN; ++a) {
                const bf16x8 yf = read_frag<TN>(yb, yfrag[a], kk);
#pragma unroll
                for (int f = 0; f < FM; ++f)
                    acc[a][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[f], yf, acc[a][f], 0, 0, 0);
            }
        }
        if constexpr (CKPT) {
            if (more) store_codes(other);
        }
        // cur's list was last read for this step's loads, ahead of the barrier above
        if (turn) store_list(then, s_tok[slot]);
        if (same) {
            i0 += BK;
            return true;
        }
        if (cur.row0 + cur.rows >= cur.end) {
            write_tile(cur);
            clear();
        }
        if (!more) return false;
        cur = nxt;
        nxt = then;
        slot ^= 1;
        i0 = 0;
        return true;
    };
    while (true) {
        if (!step(ic<0>{})) break;
        if (!step(ic<1>{})) break;
    }
}

template <int TN, int TM, bool CKPT, bool FAR>
hipError_t launch_tiles(const WgradArgs& a, hipStream_t stream) {
    static int per_cu = 0;
    if (per_cu == 0) {
        int n = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, wgrad_kernel<TN, TM, CKPT, FAR>, 512, 0) != hipSuccess || n < 1) n = 1;
        per_cu = n;
    }
    const int tn = (a.N + TN - 1) / TN, tm = (a.M + TM - 1) / TM;
    const int tiles = a.E_loc * (a.dy[1] != nullptr ? 2 : 1) * tn * tm;      // (api.hip bounds dw)
    const int most = device_cu_count() * per_cu;
    hipLaunchKernelGGL((wgrad_kernel<TN, TM, CKPT, FAR>), dim3(tiles < most ? tiles : most), dim3(512), 0, stream, a, tn, tm,
                       tiles);
    return hipGetLastError();
}

template <bool CKPT>
hipError_t launch_any(const WgradArgs& a, hipStream_t stream) {
    // direct loads reach an operand's gathered rows, or a piece's, by 32-bit offsets below kOutOfRange
    const unsigned long long y_rows = a.gather_dy ? a.src_rows : kPieceRows, x_rows = a.gather_x ? a.src_rows : kPieceRows;
    const bool far = y_rows * a.N * 2 >= (1ull << 31) || (!CKPT && x_rows * a.M * 2 >= (1ull << 31));
    if (far) return launch_tiles<256, 256, CKPT, true>(a, stream);
    const long long large = (long long)a.E_loc * (a.dy[1] != nullptr ? 2 : 1) * ((a.N + 255) / 256) * ((a.M + 255) / 256);
    if (large >= device_cu_count()) return launch_tiles<256, 256, CKPT, false>(a, stream);
    return launch_tiles<128, 128, CKPT, false>(a, stream);
}

}  // namespace

hipError_t launch_wgrad_bf16(const WgradArgs& a, hipStream_t stream) {
    return a.x_scales != nullptr ? launch_any<true>(a, stream) : launch_any<false>(a, stream);
}

}  // namespace moeep
