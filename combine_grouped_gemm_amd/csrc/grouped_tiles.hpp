// Ragged tile scheduling shared by the grouped GEMM kernels.
//
// The per-expert row counts exist only on the device (offsets of the
// contiguous layout, or the valid-row counts of the masked layout), so a
// persistent grid derives its work list there: every block builds the
// prefix sum over local experts (in id order, or most rows first) of
// ceil(rows / BM) m-tiles in LDS and maps a linear tile index tau to
// (expert j, n-tile, m-tile) by binary search, with the m-tile index fastest
// so that tiles sharing one weight tile are consecutive.  An expert's rows
// are split evenly over its m-tiles.  Blocks are renumbered XCD-major
// (hardware dispatch places block b on XCD b % 8), so consecutive tile
// indices run on one XCD and share its L2.
#pragma once

#include "device_common.hpp"
#include "launch.hpp"

namespace moeep {

constexpr int kMaxExperts = 1024;
constexpr int kXcd = 8;

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Rows [r0, r1) of local expert j: a range of the contiguous layout, or the
// first m_counts[j] rows of the expert's fixed block in the masked layout;
// both clamped to the buffer.
__device__ __forceinline__ void expert_rows(const FfnArgs& p, int j, int& r0, int& r1) {
    if (p.offsets != nullptr) {
        r0 = clampi(p.offsets[j], 0, p.cap);
        r1 = clampi(p.offsets[j + 1], r0, p.cap);
    } else {
        r0 = j * p.cap_e;
        r1 = r0 + clampi(p.m_counts[j], 0, p.cap_e);
    }
}

// Block-wide exclusive prefix into s_pre[0..n] of count(i), i in [0, n).
// s_tmp needs NT / 64 ints.  Ends with a barrier.
template <int NT, typename Count>
__device__ __forceinline__ void scan_tile_counts(int n, Count count, int* s_pre, int* s_tmp) {
    const int tid = threadIdx.x, lane = tid % kWave, wv = tid / kWave;
    constexpr int NW = NT / kWave;
    int carry = 0;
    if (tid == 0) s_pre[0] = 0;
    for (int base = 0; base < n; base += NT) {
        const int j = base + tid;
        const int v = j < n ? count(j) : 0;
        int x = v;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            int y = __shfl_up(x, d, kWave);
            if (lane >= d) x += y;
        }
        if (lane == kWave - 1) s_tmp[wv] = x;
        __syncthreads();
        int wsum = 0, total = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            wsum += (w < wv) ? s_tmp[w] : 0;
            total += s_tmp[w];
        }
        if (j < n) s_pre[j + 1] = carry + wsum + x;
        carry += total;
        __syncthreads();
    }
    __syncthreads();
}

// Block-wide exclusive prefix of m-tile counts per expert into s_pre[0..E_loc],
// experts in id order.  s_tmp needs NT / 64 ints.  Ends with a barrier.
template <int NT, int BM>
__device__ void build_tile_prefix(const FfnArgs& p, int* s_pre, int* s_tmp) {
    scan_tile_counts<NT>(p.E_loc, [&](int j) {
        int r0, r1;
        expert_rows(p, j, r0, r1);
        return (r1 - r0 + BM - 1) / BM;
    }, s_pre, s_tmp);
}

// The same prefix with the experts in decreasing row count (ties: lower id
// first): s_ord[pos] is the expert at position pos, s_pre the prefix in that
// order.  A persistent grid walks tiles in this order, so its last, partly
// filled round holds the smallest experts' tiles instead of whichever
// experts have the highest ids (longest tiles first).  s_rows is E_loc ints
// of scratch that is free at this point.  Ends with a barrier.
// BY_TILE: in decreasing row count of the experts' tiles instead (an expert of 330 rows has
// two of 165), for round_tile_back.
template <int NT, int BM, bool BY_TILE = false>
__device__ __forceinline__ void build_tile_prefix_sorted(const FfnArgs& p, int* s_pre, uint16_t* s_ord, int* s_rows,
                                         int* s_tmp) {
    const int E_loc = p.E_loc, tid = threadIdx.x;
    for (int j = tid; j < E_loc; j += NT) {
        int r0, r1;
        expert_rows(p, j, r0, r1);
        s_rows[j] = r1 - r0;
    }
    __syncthreads();
    auto key = [&](int j) {
        const int r = s_rows[j];
        if constexpr (!BY_TILE) return r;
        const int k = (r + BM - 1) / BM;
        return k > 1 ? (r + k - 1) / k : r;
    };
    for (int j = tid; j < E_loc; j += NT) {
        const int r = key(j);
        int rank = 0;
        for (int i = 0; i < E_loc; ++i) {
            const int q = key(i);
            rank += (q > r || (q == r && i < j)) ? 1 : 0;
        }
        s_ord[rank] = (uint16_t)j;
    }
    __syncthreads();
    scan_tile_counts<NT>(E_loc, [&](int pos) { return (s_rows[s_ord[pos]] + BM - 1) / BM; }, s_pre,
                         s_tmp);
}

struct TileCoord {
    int j;        // local expert
    int nt;       // n-tile
    int row0;     // first row of the tile
    int nvalid;   // valid rows in the tile (<= BM)
};

// s_ord: expert at each prefix position (build_tile_prefix_sorted), or nullptr
// for id order.
template <int BM>
__device__ __forceinline__ TileCoord decode_tile(int tau, int n_tiles_n, const int* s_pre,
                                                 const FfnArgs& p, const uint16_t* s_ord = nullptr) {
    int lo = 0, hi = p.E_loc;     // largest position j with n_tiles_n * s_pre[j] <= tau
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (n_tiles_n * s_pre[mid] <= tau) lo = mid; else hi = mid;
    }
    TileCoord t;
    t.j = s_ord != nullptr ? (int)s_ord[lo] : lo;
    const int mt_j = s_pre[lo + 1] - s_pre[lo];
    const int local = tau - n_tiles_n * s_pre[lo];
    t.nt = local / mt_j;
    const int mt = local % mt_j;
    int r0, r1;
    expert_rows(p, t.j, r0, r1);
    // balanced split: m-tile mt of mt_j takes rows [n*mt/mt_j, n*(mt+1)/mt_j) of the
    // expert, at most ceil(n/mt_j) <= BM of them
    const int n = r1 - r0;
    t.row0 = r0 + (int)(((long long)n * mt) / mt_j);
    t.nvalid = r0 + (int)(((long long)n * (mt + 1)) / mt_j) - t.row0;
    // every lane computed the same values: keep them in scalar registers, so
    // tile base addresses are scalar and stores can use 32-bit lane offsets
    t.j = __builtin_amdgcn_readfirstlane(t.j);
    t.nt = __builtin_amdgcn_readfirstlane(t.nt);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.nvalid = __builtin_amdgcn_readfirstlane(t.nvalid);
    return t;
}

// Tile of round r for the block with XCD-major position v and hardware
// index b in a grid of G, or -1 when it has none.  Rounds go in XCD-major
// order (tiles that run together are neighbours in memory and share L2),
// except a last round that fills less than half the grid: in XCD-major
// order it would run on the first few XCDs alone, so it goes in hardware
// order, spread over all of them.  (Measured on the decode-sized FFN with
// several blocks per CU: spreading a 45%-full last round 5% faster overall,
// a 78%-full one 2.7% slower.)
__device__ __forceinline__ int round_tile(int r, int v, int b, int G, int total) {
    const long long base = (long long)r * G;
    if (base >= total) return -1;
    const long long rem = total - base;
    const int tau = (int)base + (2 * rem >= G ? v : b);
    return tau < total ? tau : -1;
}

// Tile of round r for position v of G when the tiles lie in decreasing cost: every other
// round runs backwards, so that a block with a large tile of one round has a small one of
// the next (-1: none).
__device__ __forceinline__ int round_tile_back(int r, int v, int G, int total) {
    const long long tau = (long long)r * G + ((r & 1) != 0 ? G - 1 - v : v);
    return tau < total ? (int)tau : -1;
}

// Tile of the last, partly filled round: after full rounds of round_tile_back the largest tile
// left goes to the block with the least work so far (the tiles in build_tile_prefix_sorted's
// BY_TILE order, s_rows as it left them, with G more ints behind its first kMaxExperts).  A
// tile's cost: a step of wide tiles takes the time of its weights up to 128 rows and grows from
// there to 1.5 times that at 320.  Ends with a barrier.  (128 experts of 6 to 500 rows, a pair at
// 2880 x 2880, 6.3 rounds: 898 -> 879 us; gate/up of an EP share, 2.7 rounds, 581 -> 578.)
template <int NT, int BM>
__device__ __forceinline__ int last_round_tile(int full, int v, int G, int total, int n_tiles_n, int E_loc,
                                               const int* s_pre, const uint16_t* s_ord, int* s_rows, int* s_tmp) {
    const int tid = threadIdx.x;
    int* load = s_rows + kMaxExperts;
    for (int t = tid; t < G; t += NT) {
        int sum = 0;
        for (int r = 0; r < full; ++r) {
            const int tau = round_tile_back(r, t, G, total);
            int lo = 0, hi = E_loc;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (n_tiles_n * s_pre[mid] <= tau) lo = mid; else hi = mid;
            }
            const int rows = (s_rows[s_ord[lo]] + s_pre[lo + 1] - s_pre[lo] - 1) / (s_pre[lo + 1] - s_pre[lo]);
            sum += max(140, 96 + rows * 3 / 8);
        }
        load[t] = sum;
    }
    __syncthreads();
    const int mine = load[v];
    int less = 0;
    for (int t = tid; t < G; t += NT) less += load[t] < mine || (load[t] == mine && t < v) ? 1 : 0;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) less += __shfl_xor(less, d, kWave);
    if (tid % kWave == 0) s_tmp[tid / kWave] = less;
    __syncthreads();
    int rank = 0;
#pragma unroll
    for (int w = 0; w < NT / kWave; ++w) rank += s_tmp[w];
    __syncthreads();
    const int tau = __builtin_amdgcn_readfirstlane(full * G + rank);
    return tau < total ? tau : -1;
}
// rounds that last_round_tile looks back on: what it gains falls with their number
constexpr int kLookBack = 12;

// XCD-major renumbering of the block index (identity when G % 8 != 0).
__device__ __forceinline__ int xcd_block_order() {
    const int G = gridDim.x, b = blockIdx.x;
    return (G % kXcd == 0) ? (b % kXcd) * (G / kXcd) + b / kXcd : b;
}

// This block's position where there are fewer tiles than blocks: chunks of 8 (tiles that share
// weights or rows in L2) go to the XCDs in turn, whose links to memory a few tiles would
// otherwise share one of (dgrad, 7168 x 2048, 16 rows an expert: 4 experts 97 -> 81 us, 16
// experts 126 -> 94; gate/up with checkpoints of 28 experts of a few rows, 2880 -> 2880, 164 -> 155;
// with every block busy the XCD-major order is the better one, 256 rows of 32
// experts 214 us, in chunks 228).
__device__ __forceinline__ int xcd_chunk_order() {
    constexpr int kChunk = 8;
    if (gridDim.x % (kXcd * kChunk) != 0) return blockIdx.x;
    const int x = blockIdx.x % kXcd, i = blockIdx.x / kXcd;
    return i / kChunk * (kXcd * kChunk) + x * kChunk + i % kChunk;
}

template <typename Kern>
hipError_t launch_persistent(Kern kern, int threads, const FfnArgs& a, hipStream_t stream,
                             int* per_cu_cache) {
    if (*per_cu_cache == 0) {
        int n = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, 0) != hipSuccess || n < 1)
            n = 1;
        *per_cu_cache = n;
    }
    const int grid = device_cu_count() * *per_cu_cache;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(threads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace moeep
