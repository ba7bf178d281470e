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
// and the tile's stores drain under the next tile's steps.  32 experts of 85 to 1026 rows, a pair of
// 2048 x 7168 in fp32 from a checkpoint: 1110 us, 3.76 GB of dw at 3.4 TB/s (in bf16 844 us); with
// a base, 2.12 GB at 2880 x 2880, 444 us, the rate of a copy.  256 CUs that do nothing but store
// such tiles reach 5.5 TB/s, and a load waits behind the stores of all of its CU's waves, not only
// its own's (stores alone 384 us, loads alone 98, both 469), so deeper rings, waves that only
// load and blocks side by side do not help: a ring of four 32-row stages 1057 us where this
// takes 900, two 128 x 128 blocks a CU 1549.
//
// The row of a gathered operand (src_of) is looked up once per piece of work (a tile, or
// 1024 rows of one): the piece's rows are listed in LDS during the piece before, so that a
// load's address is one LDS read away.  Rows past the expert's last one get an offset outside
// the operand's extent, read nothing and land zeros in both operands.  So do rows of the gathered
// operand that src_of names nowhere; a list says whether it has any, and then their rows of the
// other operand are cleared in LDS, so that they add nothing whatever it holds.  (The EP
// share above, one set of operands: with no such list 1045 us, so 1063, with both operands'
// offsets from the list 1080.)
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
// Offsets out of range: kOutOfRange for a row, this for a column.  A sum of the two, or of
// either and an offset below kReach, stays below 2^32 and at or above kReach, which every
// extent stays under.
constexpr uint32_t kNoColumn = 0x7fff0000u;
constexpr unsigned long long kReach = kNoColumn;

constexpr int kGroup = 4;                    // tiles along the in columns that are done together

#define INLINE __attribute__((always_inline))

// what a lane of a 64-bit load reads where there is nothing to read
__device__ uint4 g_zeros;

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
template <int CPOL>
__device__ __forceinline__ uint4 buf_load16(rsrc_t r, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, CPOL));
#else
    return make_uint4(0, 0, 0, 0);
#endif
}
__device__ __forceinline__ float buf_load4(rsrc_t r, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
#else
    return 0.0f;
#endif
}
template <int CPOL>
__device__ __forceinline__ void buf_store16(rsrc_t r, uint32_t off, uint4 v) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, (int)off, 0, CPOL);
#endif
}

// a piece of work: rows [row0, row0 + rows) of a tile's expert
struct Piece {
    int tile, j, q, n0, m0, row0, rows, end;     // end: the expert's last row, exclusive
};

// TN, TM: tile of dw (out x in); 8 waves, 2 (out) x 4 (in).  FAR: an operand, or a tile's
// rows of dw, that 32-bit offsets do not reach: 64-bit addresses.
template <int TN, int TM, bool CKPT, bool F32, bool FAR>
__global__ __launch_bounds__(512, 1) void wgrad_kernel(WgradArgs p, int tiles_n, int tiles_m, int tiles) {
    constexpr int NT = 512, NW = 8;
    constexpr int FN = TN / 2 / 16, FM = TM / 4 / 16;        // fragments of a wave
    constexpr int Y_ITERS = BK * TN * 2 / 1024 / NW;         // direct loads of a wave per step
    constexpr int X_ITERS = BK * TM * 2 / 1024 / NW;
    constexpr int C_ITERS = BK * TM / 1024 / NW;             // checkpoint: 16-code loads of a lane
    constexpr int YR = 512 / TN, XR = 512 / TM;              // rows of a direct load
    constexpr int CR = 1024 / TM;                            // rows of a wave's code load
    constexpr int LOADS = Y_ITERS + (CKPT ? 0 : X_ITERS);
    // dw in 16-byte units: 4 columns of fp32, 8 of bf16
    constexpr int SIZE = F32 ? 4 : 2, WIDE = 16 / SIZE, UNITS = FM * 4 / WIDE;
    constexpr int STORES = FN * UNITS;                       // of a wave and tile, whatever its borders
    static_assert(Y_ITERS >= 1 && X_ITERS >= 1 && C_ITERS >= 1 && STORES < 64, "tile shape");

    // each stage an object of its own: the compiler sees that reads of one do not
    // depend on the loads in flight into the other
    __shared__ uint4 sy0[BK * TN / 8];
    __shared__ uint4 sx0[BK * TM / 8];
    __shared__ uint4 sy1[BK * TN / 8];
    __shared__ uint4 sx1[BK * TM / 8];
    __shared__ int s_tok[2][kPieceRows];
    __shared__ uint2 s_holes[2];                             // whether a list has such a row (a byte a wave)
    __shared__ int s_off[kMaxExperts + 1];                   // the experts' offsets, within the buffer

    auto y_base = [&](auto I) INLINE -> char* {
        if constexpr (decltype(I)::value == 0) return reinterpret_cast<char*>(sy0);
        else return reinterpret_cast<char*>(sy1);
    };
    auto x_base = [&](auto I) INLINE -> char* {
        if constexpr (decltype(I)::value == 0) return reinterpret_cast<char*>(sx0);
        else return reinterpret_cast<char*>(sx1);
    };

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = uniform(tid / kWave);
    const int wn = wave / 4, wm = wave % 4;
    const int N = p.N, M = p.M, G = gridDim.x;
    const int nb = (M + kCkptBlock - 1) / kCkptBlock;
    const bool gathers = p.src_of != nullptr;

    auto open_tile = [&](int tau, Piece& w) INLINE {
        w.tile = tau;
        w.row0 = w.rows = w.end = 0;
        if (tau >= tiles) return;
        // Groups of kGroup tiles along the in columns, within them all tiles along the out
        // columns, then the pair: the 32 tiles that run together on an XCD share 8 + 4 operand
        // columns of tiles in its L2, and the next ones go on with the 4.
        const unsigned pairs = p.dw[1] != nullptr ? 2 : 1, per = (unsigned)tiles_n * (unsigned)tiles_m * pairs;
        w.j = uniform((int)((unsigned)tau / per));
        unsigned rest = (unsigned)tau - (unsigned)w.j * per;
        const unsigned band = (unsigned)tiles_n * kGroup * pairs, b = rest / band;
        rest -= b * band;
        const unsigned wide = min((unsigned)tiles_m - b * kGroup, (unsigned)kGroup), one = (unsigned)tiles_n * wide;
        w.q = uniform(rest >= one ? 1 : 0);
        rest -= w.q ? one : 0u;
        const unsigned n = rest / wide;
        w.n0 = uniform((int)n * TN);
        w.m0 = uniform((int)(b * kGroup + rest - n * wide) * TM);
        w.row0 = uniform(s_off[w.j]);
        w.end = uniform(max(s_off[w.j + 1], w.row0));
        w.rows = min(w.end - w.row0, kPieceRows);
    };
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
    // the slots of a piece's rows, and the list of the rows that a gathered operand reads for
    // them (-1: none, also behind the last row)
    constexpr int LIST = kPieceRows / NT;
    int listed[LIST];
    auto load_list = [&](const Piece& w) INLINE {
        if (!gathers) return;
#pragma unroll
        for (int i = 0; i < LIST; ++i) {
            const int r = i * NT + tid;
            listed[i] = r < w.rows ? p.src_of[w.row0 + r] : -1;
        }
    };
    auto store_list = [&](const Piece& w, int list) INLINE {
        if (!gathers) return;
        bool hole = false;
#pragma unroll
        for (int i = 0; i < LIST; ++i) {
            const int r = i * NT + tid;
            int t = listed[i] < 0 ? -1 : token_of(listed[i], p.per_div);
            t = t < p.src_rows ? t : -1;
            s_tok[list][r] = t;
            hole |= t < 0 && r < w.rows;
        }
        const bool any = ballot64(hole) != 0;
        if (lane == 0) reinterpret_cast<uint8_t*>(&s_holes[list])[wave] = any;
    };

    // What a step of piece w that starts at its row i0 loads.  Lane offsets of the direct
    // loads: a gathered row lies anywhere in its operand, another is counted from the step's
    // first one and the extent ends with the piece's rows.
    uint32_t yoff[Y_ITERS], xoff[X_ITERS];
    int yrow[Y_ITERS], xrow[X_ITERS];                         // FAR: the rows themselves
    auto operand_rows = [&](auto iters, auto rows_of, bool gathered, int pitch, int c0, int width, const Piece& w,
                            const int* tok, int i0, uint32_t* off, int* row) INLINE {
        constexpr int ITERS = decltype(iters)::value, R = decltype(rows_of)::value, T = 512 / R;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int k = (i * NW + wave) * R + lane / (64 / R);
            const int col = c0 + ((lane % (64 / R)) ^ swz_row<T>(k)) * 8;
            const uint32_t cb = col < width ? (uint32_t)col * 2 : kNoColumn;
            int r = k;
            if (gathered) r = tok[i0 + k];
            if constexpr (FAR) {
                row[i] = gathered ? r : (i0 + k < w.rows ? w.row0 + i0 + k : -1);
                off[i] = cb;
            } else {
                off[i] = (r >= 0 ? (uint32_t)r * (uint32_t)pitch : kOutOfRange) + cb;
            }
        }
    };
    struct Source {
        rsrc_t y, x;
        const char *ybase, *xbase;
    };
    auto issue_y = [&](auto I, const Source& s, int i) INLINE {
        char* dst = y_base(I) + (i * NW + wave) * 1024;
        if constexpr (FAR)
            lds_dma16<0>(yrow[i] >= 0 && yoff[i] != kNoColumn ? s.ybase + (size_t)yrow[i] * N * 2 + yoff[i]
                                                             : reinterpret_cast<const char*>(&g_zeros), dst);
        else
            lds_buf16<0>(s.y, dst, yoff[i], 0);
    };
    auto issue_x = [&](auto I, const Source& s, int i) INLINE {
        char* dst = x_base(I) + (i * NW + wave) * 1024;
        if constexpr (FAR)
            lds_dma16<0>(xrow[i] >= 0 && xoff[i] != kNoColumn ? s.xbase + (size_t)xrow[i] * M * 2 + xoff[i]
                                                             : reinterpret_cast<const char*>(&g_zeros), dst);
        else
            lds_buf16<0>(s.x, dst, xoff[i], 0);
    };
    // 16 codes of a row and their scale; zeros where there is no row.  A row that ends with 8
    // codes reads 8 of the next one, in columns that dw does not have.
    uint4 code[C_ITERS];
    float cscale[C_ITERS];
    auto load_codes = [&](const Piece& w, const int* tok, int i0) INLINE {
        const int rows = p.gather_x ? p.src_rows : p.cap;
#pragma unroll
        for (int i = 0; i < C_ITERS; ++i) {
            const int k = (i * NW + wave) * CR + lane / (TM / 16);
            const int col = w.m0 + (lane % (TM / 16)) * 16;
            int r = i0 + k < w.rows ? w.row0 + i0 + k : -1;
            if (p.gather_x) r = tok[i0 + k];
            const bool here = r >= 0 && col < M;
            if constexpr (FAR) {
                code[i] = make_uint4(0, 0, 0, 0);
                cscale[i] = 0.0f;
                if (here) {
                    const int8_t* row = static_cast<const int8_t*>(p.x) + (size_t)r * M + col;
                    const uint2 lo = *reinterpret_cast<const uint2*>(row);
                    const uint2 hi = col + 8 < M ? *reinterpret_cast<const uint2*>(row + 8) : make_uint2(0, 0);
                    code[i] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                    cscale[i] = p.x_scales[(size_t)r * nb + col / kCkptBlock];
                }
            } else {
                code[i] = buf_load16<0>(make_rsrc(p.x, (uint32_t)rows * (uint32_t)M),
                                     here ? (uint32_t)r * (uint32_t)M + (uint32_t)col : kOutOfRange);
                cscale[i] = buf_load4(make_rsrc(p.x_scales, (uint32_t)rows * (uint32_t)nb * 4u),
                                      here ? ((uint32_t)r * (uint32_t)nb + (uint32_t)(col / kCkptBlock)) * 4u : kOutOfRange);
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
    // zeros in both operands' rows that src_of names nowhere, in a stage whose loads have landed
    auto clear_holes = [&](auto I, const int* tok) INLINE {
        for (int k = wave; k < BK; k += NW) {
            if (uniform(tok[k]) >= 0) continue;
            for (int c = lane; c < TN / 8; c += kWave)
                reinterpret_cast<uint4*>(y_base(I))[k * (TN / 8) + c] = make_uint4(0, 0, 0, 0);
            for (int c = lane; c < TM / 8; c += kWave)
                reinterpret_cast<uint4*>(x_base(I))[k * (TM / 8) + c] = make_uint4(0, 0, 0, 0);
        }
        wait_lgkm0();
        block_barrier();
    };
    // everything that precedes the direct loads of a step
    auto prepare = [&](const Piece& w, const int* tok, int i0, bool live) INLINE {
        Source s;
        if constexpr (CKPT) load_codes(w, tok, i0);
        operand_rows(ic<Y_ITERS>{}, ic<YR>{}, p.gather_dy, N * 2, w.n0, N, w, tok, i0, yoff, yrow);
        if constexpr (!CKPT) operand_rows(ic<X_ITERS>{}, ic<XR>{}, p.gather_x, M * 2, w.m0, M, w, tok, i0, xoff, xrow);
        const char* dy = static_cast<const char*>(w.q == 0 ? p.dy[0] : p.dy[1]);
        if constexpr (FAR) {
            s.ybase = dy;
            s.xbase = static_cast<const char*>(p.x);
        } else {
            const uint32_t left = live ? (uint32_t)(w.rows - i0) : 0u, all = live ? (uint32_t)p.src_rows : 0u;
            s.y = p.gather_dy ? make_rsrc(dy, all * (uint32_t)(N * 2))
                              : make_rsrc(dy + (size_t)(w.row0 + i0) * N * 2, left * (uint32_t)(N * 2));
            if constexpr (!CKPT) {
                const char* x = static_cast<const char*>(p.x);
                s.x = p.gather_x ? make_rsrc(x, all * (uint32_t)(M * 2))
                                 : make_rsrc(x + (size_t)(w.row0 + i0) * M * 2, left * (uint32_t)(M * 2));
            }
        }
        return s;
    };

    const uint32_t yfrag0 = frag_offset<TN>(lane, wn * (FN * 16)), xfrag0 = frag_offset<TM>(lane, wm * (FM * 16));

    floatx4 acc[FN][FM];
    auto clear = [&]() INLINE {
#pragma unroll
        for (int a = 0; a < FN; ++a)
#pragma unroll
            for (int b = 0; b < FM; ++b) acc[a][b] = floatx4{0.f, 0.f, 0.f, 0.f};
    };
    clear();

    // dw of a finished tile.  Lane l of a fragment has row n = l % 16 and columns 4 (l / 16) ..
    // + 3.  Lanes exchange values so that a unit is 16 bytes and a store covers whole 128-byte
    // lines (8 rows of them; bf16 in 128-column tiles half lines): such stores can be
    // non-temporal, and dw, 117 MB a pair in fp32 at 2048 x 7168, does not push the operands out of L2.
    // (Half lines, kept in L2: EP share 1509 us; whole ones, not kept, 1238 us.)  All stores go
    // out, those past the borders to an offset out of range, so that their number is known to
    // the wait of the next step.  A base is read one row of fragments ahead of the stores.
    const int g = lane >> 4, n8 = lane & 7, upper = (lane >> 3) & 1;
    auto unit_row = [&](int u) INLINE { return n8 + (F32 ? (u & 1) * 8 : FM == 4 ? u * 8 : (g & 1) * 8); };
    auto unit_col = [&](int u) INLINE {
        return upper * 16 + (F32 ? (u >> 1) * 32 + g * 4 : (FM == 4 ? (g & 1) * 32 : 0) + (g >> 1) * 8);
    };
    auto units_of = [&](int a, float (&v)[UNITS][WIDE]) INLINE {
        float t[FM][4];
#pragma unroll
        for (int f = 0; f < FM; f += 2)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                t[f][e] = acc[a][f][e];
                t[f + 1][e] = acc[a][f + 1][e];
                exchange_rows(t[f][e], t[f + 1][e]);
            }
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (F32) v[u][e] = t[u][e];
                else {
                    // rows 8 u .. + 7 of both column pairs; of the only pair, rows 0..7 and 8..15
                    float x = t[u][e], y = t[FM == 4 ? u + 2 : 1][e];
                    exchange_groups(x, y);
                    v[u][e] = x;
                    v[u][4 + e] = y;
                }
            }
    };
    auto write_as = [&](const Piece& w, bool based) INLINE {
        const size_t at = ((size_t)w.j * N + w.n0) * M * SIZE;
        const char* base = static_cast<const char*>(w.q == 0 ? p.base[0] : p.base[1]) + at;
        char* dw = static_cast<char*>(w.q == 0 ? p.dw[0] : p.dw[1]) + at;
        const int m = w.m0 + wm * (FM * 16), n = wn * (FN * 16);
        const uint32_t bytes = FAR ? 0u : (uint32_t)min(TN, N - w.n0) * (uint32_t)M * SIZE, pitch = (uint32_t)M * SIZE;
        const rsrc_t rw = make_rsrc(dw, bytes), rb = make_rsrc(base, based ? bytes : 0u);
        uint32_t off[UNITS];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int col = m + unit_col(u);
            off[u] = (col < M ? (uint32_t)col * SIZE : kNoColumn) + (uint32_t)(n + unit_row(u)) * pitch;
        }
        constexpr int CPOL = F32 || FM == 4 ? kNonTemporal : 0;
        uint4 b[2][UNITS];
        auto load_base = [&](int a) INLINE {
#pragma unroll
            for (int u = 0; u < UNITS; ++u) b[a & 1][u] = buf_load16<CPOL>(rb, off[u] + a * 16 * pitch);
        };
        if (!FAR && based) load_base(0);
#pragma unroll
        for (int a = 0; a < FN; ++a) {
            if (!FAR && based && a + 1 < FN) load_base(a + 1);
            float v[UNITS][WIDE];
            units_of(a, v);
#pragma unroll
            for (int u = 0; u < UNITS; ++u) {
                const int row = n + a * 16 + unit_row(u), col = m + unit_col(u);
                const bool here = w.n0 + row < N && col < M;
                const size_t o = ((size_t)row * M + col) * SIZE;
                if (based) {
                    if constexpr (FAR) b[a & 1][u] = here ? *reinterpret_cast<const uint4*>(base + o) : make_uint4(0, 0, 0, 0);
                    const uint32_t t[4] = {b[a & 1][u].x, b[a & 1][u].y, b[a & 1][u].z, b[a & 1][u].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (F32) v[u][e] += __uint_as_float(t[e]);
                        else {
                            v[u][2 * e] += bf16_lo(t[e]);
                            v[u][2 * e + 1] += bf16_hi(t[e]);
                        }
                    }
                }
                uint4 t;
                if constexpr (F32)
                    t = make_uint4(__float_as_uint(v[u][0]), __float_as_uint(v[u][1]), __float_as_uint(v[u][2]),
                                   __float_as_uint(v[u][3]));
                else
                    t = make_uint4(pack_bf16x2(v[u][0], v[u][1]), pack_bf16x2(v[u][2], v[u][3]),
                                   pack_bf16x2(v[u][4], v[u][5]), pack_bf16x2(v[u][6], v[u][7]));
                if constexpr (FAR) {
                    if (here) *reinterpret_cast<uint4*>(dw + o) = t;
                } else {
                    buf_store16<CPOL>(rw, off[u] + a * 16 * pitch, t);
                }
            }
        }
    };
    auto write_tile = [&](const Piece& w) INLINE {
        if ((w.q == 0 ? p.base[0] : p.base[1]) != nullptr) write_as(w, true);
        else write_as(w, false);
    };

    // (read here once: a load in the sequence of steps would wait for the stores before it)
    for (int j = tid; j <= p.E_loc; j += NT) s_off[j] = clampi(p.offsets[j], 0, p.cap);
    __syncthreads();

    // the sequence of steps: `cur` is computed, `nxt` comes after it; s_tok[slot] lists cur's rows
    Piece cur, nxt, then;
    cur.j = cur.q = cur.n0 = cur.m0 = 0;
    open_tile(xcd_block_order(), cur);
    if (cur.tile >= tiles) return;
    load_list(cur);
    store_list(cur, 0);
    nxt = after(cur);
    load_list(nxt);
    store_list(nxt, 1);
    __syncthreads();
    {
        const Source s = prepare(cur, s_tok[0], 0, true);
#pragma unroll
        for (int i = 0; i < Y_ITERS; ++i) issue_y(ic<0>{}, s, i);
        if constexpr (CKPT) store_codes(ic<0>{});
        else {
#pragma unroll
            for (int i = 0; i < X_ITERS; ++i) issue_x(ic<0>{}, s, i);
        }
    }
    int slot = 0, i0 = 0;                        // i0: first row of cur's step
    bool draining = false;                                   // a tile's stores are the last things issued

    // one step; false after the last one of all
    auto step = [&](auto I) INLINE -> bool {
        const uint2 holes = s_holes[slot];
        // this step's loads have landed; a tile's stores issued after them may still be on their way
        if (draining) wait_vmcnt<STORES>();
        else wait_vmcnt<0>();
        draining = false;
        wait_lgkm0();
        block_barrier();
        if (gathers && uniform((int)(holes.x | holes.y)) != 0) clear_holes(I, s_tok[slot] + i0);
        // what comes next: another step of this piece, or the first of the next piece
        const bool same = uniform(i0 + BK < cur.rows ? 1 : 0) != 0;
        const bool more = uniform(same || nxt.tile < tiles ? 1 : 0) != 0;
        const bool turn = uniform(!same && more ? 1 : 0) != 0;
        if (turn) {
            then = after(nxt);
            load_list(then);
        }
        {
            constexpr auto other = ic<1 - decltype(I)::value>{};
            const Piece& w = same ? cur : nxt;
            // (past the last step nothing is read, but the loads go out)
            const Source s = prepare(w, s_tok[same ? slot : slot ^ 1], same ? i0 + BK : 0, more);
            // fragments come in blocks of four, read and waited for together: the compiler, left to
            // place the waits, lets a read wait for every load and store in flight
            uint32_t ya[FN], xa[FM];
#pragma unroll
            for (int a = 0; a < FN; ++a) ya[a] = lds_addr(y_base(I)) + (yfrag0 ^ (a << 5));
#pragma unroll
            for (int f = 0; f < FM; ++f) xa[f] = lds_addr(x_base(I)) + (xfrag0 ^ (f << 5));
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                bf16x8 xf[FM];
                if (kk == 0) read_frags<TM, 0>(xf, xa);
                else read_frags<TM, 1>(xf, xa);
#pragma unroll
                for (int a0 = 0; a0 < FN; a0 += 4) {
                    bf16x8 yf[4];
                    const uint32_t ad[4] = {ya[a0], ya[a0 + 1], ya[a0 + 2], ya[a0 + 3]};
                    if (kk == 0) read_frags<TN, 0>(yf, ad);
                    else read_frags<TN, 1>(yf, ad);
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
#pragma unroll
                        for (int f = 0; f < FM; ++f)
                            acc[a0 + a][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[f], yf[a], acc[a0 + a][f], 0, 0, 0);
                        const int q = kk * FN + a0 + a;
                        if (q < Y_ITERS) issue_y(other, s, q);
                        else if (q < LOADS) issue_x(other, s, q - Y_ITERS);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
#pragma unroll
            for (int q = 2 * FN; q < LOADS; ++q) {
                if (q < Y_ITERS) issue_y(other, s, q);
                else issue_x(other, s, q - Y_ITERS);
            }
            if constexpr (CKPT) store_codes(other);
        }
        // cur's list was last read for this step's loads, ahead of the barrier above
        if (turn) store_list(then, slot);
        if (same) {
            i0 += BK;
            return true;
        }
        if (cur.row0 + cur.rows >= cur.end) {
            write_tile(cur);
            clear();
            draining = !FAR;
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
    wait_vmcnt<0>();                                         // the loads past the last step have landed
}

template <int TN, int TM, bool CKPT, bool F32, bool FAR>
hipError_t launch_tiles(const WgradArgs& a, hipStream_t stream) {
    static int per_cu = 0;
    if (per_cu == 0) {
        int n = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, wgrad_kernel<TN, TM, CKPT, F32, FAR>, 512, 0) != hipSuccess || n < 1) n = 1;
        per_cu = n;
    }
    const int tn = (a.N + TN - 1) / TN, tm = (a.M + TM - 1) / TM;
    const int tiles = a.E_loc * (a.dw[1] != nullptr ? 2 : 1) * tn * tm;      // (api.hip bounds dw)
    const int most = device_cu_count() * per_cu;
    hipLaunchKernelGGL((wgrad_kernel<TN, TM, CKPT, F32, FAR>), dim3(tiles < most ? tiles : most), dim3(512), 0, stream, a, tn, tm,
                       tiles);
    return hipGetLastError();
}

template <bool CKPT, bool F32>
hipError_t launch_any(const WgradArgs& a, hipStream_t stream) {
    // 32-bit offsets reach an operand's gathered rows (others: a piece's), all codes and scales,
    // and a tile's rows of dw
    const unsigned long long y_rows = a.gather_dy ? a.src_rows : kPieceRows;
    const unsigned long long x_rows = a.gather_x ? a.src_rows : CKPT ? a.cap : kPieceRows;
    const bool far = y_rows * a.N * 2 >= kReach || x_rows * a.M * (CKPT ? 1 : 2) >= kReach || 256ull * a.M * 4 >= kReach;
    // (64-bit addresses where not needed: 32 experts of 256 rows, 2048 x 7168, 575 us beside 456, one
    // set of operands that stays in the Infinity Cache; of several sets 578 for those 456)
    if (far) return launch_tiles<256, 256, CKPT, F32, true>(a, stream);
    // large tiles once there is one for every CU: that case 456 us, in small ones 525; 8 experts of
    // 64 rows, 1024 x 1024 (128 large tiles) 15.3, small 13.1; 4 of 512 rows, 512 x 512, 25.4 and 13.0
    const long long large = (long long)a.E_loc * (a.dw[1] != nullptr ? 2 : 1) * ((a.N + 255) / 256) * ((a.M + 255) / 256);
    if (large >= device_cu_count()) return launch_tiles<256, 256, CKPT, F32, false>(a, stream);
    return launch_tiles<128, 128, CKPT, F32, false>(a, stream);
}

}  // namespace

hipError_t launch_wgrad_bf16(const WgradArgs& a, hipStream_t stream) {
    if (a.dw_f32) return a.x_scales != nullptr ? launch_any<true, true>(a, stream) : launch_any<false, true>(a, stream);
    return a.x_scales != nullptr ? launch_any<true, false>(a, stream) : launch_any<false, false>(a, stream);
}

}  // namespace moeep
