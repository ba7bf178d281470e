// Per-row int8 quantisation: of the tokens on their way to the experts
// (dispatch) and of expert-ordered rows (h between gate/up and down; weight
// rows, i.e. output channels).
//
// For a row v: amax = max |v|, scale = RN(amax / 127) in fp32 (at least the
// smallest normal number; 1 for amax = 0), code = v / scale rounded to the
// nearest integer, ties to even.  The quotient is rounded exactly: n =
// RN(v * RN(1 / scale)) is off by at most one step, and only next to a tie,
// and the remainder v - n * scale is exact in one fma (v and scale share the
// 24-bit grid of the larger one's last place, and |remainder| <= 0.51 scale),
// so comparing it with scale / 2 settles the code.  A row with a NaN or an
// infinity gets scale NaN and codes 0: every product with it is NaN.
//
// Both kernels move data and little else: the row is read once into registers
// (16 consecutive values a lane and piece: 32 bytes of bf16 in, 16 bytes of
// codes out), reduced, quantised and stored.  n comes from one fma onto 1.5 *
// 2^23, whose low byte is the code; a piece is done again by the long way only
// if one of its remainders reaches half a step (a row in fifty at 2048
// columns).  About six instructions an element, a third of the time that its
// three bytes take at the rate of a large copy.
//
// Measured (MI355X, in a graph): 65536 rows of 2048 bf16 values 80 us, 5.0 TB/s
// (a large copy: 4.9; reading each row twice 95 us); 1024 rows in 256 blocks of
// 32, from cold caches, 6.1 us.  Dispatch of one EP=8 rank's share, 3684 tokens of 7168: 14-15 us,
// 4.2 TB/s (21 us with two reads), 19 us from cold caches; 128 tokens to 8 rows
// each 5.7 us (8.0).
#include "device_common.hpp"
#include "launch.hpp"

namespace moeep {
namespace {

// Scale of a row whose largest magnitude has the bits `amax` (sign cleared).
__device__ __forceinline__ float row_scale(uint32_t amax) {
    if (amax == 0u) return 1.0f;
    if (amax >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    return fmaxf(__uint_as_float(amax) / 127.0f, 1.17549435e-38f);
}

// Code of v for the row scale s, rs = 1 / s (see the file comment).
__device__ __forceinline__ int code_of(float v, float s, float rs) {
    float n = rintf(v * rs);
    const float r = fmaf(-n, s, v), h = 0.5f * s;
    const bool odd = ((int)n & 1) != 0;
    if (r > h || (r == h && odd)) n += 1.0f;
    else if (r < -h || (r == -h && odd)) n -= 1.0f;
    return (int)n;
}

// 16 consecutive values of a row, as they are in memory: 32 bytes of bf16 or 64 of fp32.
template <bool F32>
struct Piece {
    static constexpr int kVec = F32 ? 4 : 2;
    uint4 v[kVec];

    __device__ __forceinline__ void load(const void* row, int c) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = static_cast<const uint4*>(row)[c * kVec + i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void values(float (&f)[16]) const {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (F32) f[i * 4 + k] = __uint_as_float(w[k]);
                else {
                    f[i * 8 + k * 2] = bf16_lo(w[k]);
                    f[i * 8 + k * 2 + 1] = bf16_hi(w[k]);
                }
            }
        }
    }
    __device__ __forceinline__ uint32_t amax(uint32_t m) const {
        float f[16];
        values(f);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t u = __float_as_uint(f[i]) & 0x7fffffffu;
            m = u > m ? u : m;
        }
        return m;
    }
    // the 16 codes; s NaN: zeros
    __device__ __forceinline__ uint4 codes(float s, float rs) const {
        float f[16];
        values(f);
        constexpr float kMagic = 12582912.0f;                    // 1.5 * 2^23
        uint32_t t[16], q[4];
        float far = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float m = fmaf(f[i], rs, kMagic);
            far = fmaxf(far, fabsf(fmaf(kMagic - m, s, f[i])));
            t[i] = __float_as_uint(m);
        }
        if (far >= 0.5f * s) {
#pragma unroll
            for (int i = 0; i < 16; ++i) t[i] = (uint32_t)code_of(f[i], s, rs);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = __builtin_amdgcn_perm(t[i * 4 + 1], t[i * 4], 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(t[i * 4 + 3], t[i * 4 + 2], 0x04000c0cu);
            q[i] = s == s ? lo | hi : 0u;
        }
        return make_uint4(q[0], q[1], q[2], q[3]);
    }
};

// Maximum over the wave, the same in every lane: within each 16-lane row by
// DPP (partners lane ^ 1, lane ^ 2, then the half-row and row mirrors), then
// over one lane of each row.  As integers: bit patterns of magnitudes, NaN above
// everything.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    auto most = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    v = most(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
    v = most(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
    v = most(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));
    v = most(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));
    const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0), b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
    const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32), d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
    return most(most(a, b), most(c, d));
}

// ---- dispatch: one block per token, its pieces spread over the threads, NP
// to each (0: any number, read a second time from cache for the codes).  The
// token's destination rows come with one vector load per wave (lane k holds
// slot k's row; a ballot gives the local slots), as in dispatch.hip; a token
// without a local slot is not read.
constexpr int kTokThreads = 512;             // most threads per block

__device__ __forceinline__ int slot_row(const int32_t* rows, int K, int k0, int cap, int lane) {
    const int k = k0 + lane;
    if (k >= K) return -1;
    const int r = rows[k];
    return (r >= 0 && r < cap) ? r : -1;
}

template <bool F32, int NP>
__global__ __launch_bounds__(kTokThreads) void dispatch_i8_kernel(
    SegTable seg, int H, const int32_t* __restrict__ row_of, int K, int cap, uint8_t* __restrict__ xd,
    float* __restrict__ xd_scales) {
    __shared__ uint32_t s_max[kTokThreads / kWave];
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid % kWave, nt = blockDim.x, np = H / 16;
    const int32_t* rows = row_of + (size_t)t * K;
    int my = slot_row(rows, K, 0, cap, lane);
    uint64_t local = ballot64(my >= 0);       // local slots among the first 64, the same in every wave
    bool any = local != 0;
    for (int k0 = kWave; k0 < K && !any; k0 += kWave) any = ballot64(slot_row(rows, K, k0, cap, lane) >= 0) != 0;
    if (!any) return;
    int i = 0;                                // the token's segment
    for (int s = 1; s < seg.n; ++s) i += t >= seg.start[s] ? 1 : 0;
    const char* row = static_cast<const char*>(seg.ptr[i]) + (size_t)(t - seg.start[i]) * H * (F32 ? 4 : 2);

    constexpr int kHeld = NP > 0 ? NP : 1;
    Piece<F32> piece[kHeld];
    uint32_t m = 0;
    if constexpr (NP > 0) {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const int c = tid + n * nt;
            if (c < np) piece[n].load(row, c);
            else piece[n].zero();
        }
#pragma unroll
        for (int n = 0; n < NP; ++n) m = piece[n].amax(m);
    } else {
        for (int c = tid; c < np; c += nt) {
            piece[0].load(row, c);
            m = piece[0].amax(m);
        }
    }
    m = wave_max_u32(m);
    if (nt > kWave) {
        if (lane == 0) s_max[tid / kWave] = m;
        __syncthreads();
        for (int w = 0; w < nt / kWave; ++w) m = s_max[w] > m ? s_max[w] : m;
    }
    const float s = row_scale(m), rs = 1.0f / s;
    if constexpr (NP > 0) {
        uint4 q[NP];
#pragma unroll
        for (int n = 0; n < NP; ++n) q[n] = piece[n].codes(s, rs);
        for (int k0 = 0;;) {
            if (my >= 0 && tid < kWave) xd_scales[my] = s;
            while (local != 0) {
                const int k = __builtin_ctzll(local);
                local &= local - 1;
                uint4* dst = reinterpret_cast<uint4*>(xd + (size_t)__builtin_amdgcn_readlane(my, k) * H);
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    const int c = tid + n * nt;
                    if (c < np) dst[c] = q[n];
                }
            }
            k0 += kWave;
            if (k0 >= K) break;
            my = slot_row(rows, K, k0, cap, lane);
            local = ballot64(my >= 0);
        }
    } else {
        for (int k = tid; k < K; k += nt) {
            const int r = rows[k];
            if (r >= 0 && r < cap) xd_scales[r] = s;
        }
        for (int c = tid; c < np; c += nt) {
            piece[0].load(row, c);
            const uint4 q = piece[0].codes(s, rs);
            for (int k = 0; k < K; ++k) {
                const int r = rows[k];
                if (r >= 0 && r < cap) reinterpret_cast<uint4*>(xd + (size_t)r * H)[c] = q;
            }
        }
    }
}

// ---- expert-ordered rows.  Valid rows are [offsets[0], offsets[E_loc]) of the
// contiguous layout or all rows: a persistent grid walks them.  In the masked
// layout (the first m[j] rows of each block of cap_e) blockIdx.y is the expert,
// and its blocks share its rows.  A row goes to a wave or to a block of four,
// whichever hides the row's latency better: short rows (up to 1024 columns) to a
// wave, long ones (over 4096) to a block, those between to a block while there
// are few of them (`few`, of the layout or of the expert; the device knows how
// many there are).  Measured, us, wave against block, 256 / 4096 / 16384 rows of
// bf16: 1024 columns 3.4 / 5.4 / 12.7, 3.3 / 8.6 / 27.3; 2048 5.3 / 9.2 / 21.2,
// 3.4 / 10.5 / 31.9; 4096 8.6 / 15.8 / 41.9, 4.1 / 13.0 / 40.7; 8192 14.0 / 29.3 /
// 90.5, 6.4 / 21.9 / 83.9.  At 2048 columns they meet at 2048 rows (6.7, 6.2).
constexpr int kRowWaves = 4;

// t: this thread among the row's W waves; s_max: W words of LDS that no other wave
// still reads
template <bool F32, int NP, int W>
__device__ __forceinline__ void quant_row(const QuantArgs& p, size_t r, int t, uint32_t* s_max) {
    constexpr int kStride = W * kWave;
    const char* row = static_cast<const char*>(p.x) + r * p.cols * (F32 ? 4 : 2);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.q) + r * p.cols);
    const int np = p.cols / 16;
    constexpr int kHeld = NP > 0 ? NP : 1;
    Piece<F32> piece[kHeld];
    uint32_t m = 0;
    if constexpr (NP > 0) {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const int c = t + n * kStride;
            if (c < np) piece[n].load(row, c);
            else piece[n].zero();
        }
#pragma unroll
        for (int n = 0; n < NP; ++n) m = piece[n].amax(m);
    } else {
        for (int c = t; c < np; c += kStride) {
            piece[0].load(row, c);
            m = piece[0].amax(m);
        }
    }
    m = wave_max_u32(m);
    if constexpr (W > 1) {
        if (t % kWave == 0) s_max[t / kWave] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) m = s_max[w] > m ? s_max[w] : m;
    }
    const float s = row_scale(m), rs = 1.0f / s;
    if constexpr (NP > 0) {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const int c = t + n * kStride;
            const uint4 q = piece[n].codes(s, rs);
            if (c < np) dst[c] = q;
        }
    } else {
        for (int c = t; c < np; c += kStride) {
            piece[0].load(row, c);
            dst[c] = piece[0].codes(s, rs);
        }
    }
    if (t == 0) p.scales[r] = s;
}

// WAVE, BLOCK: pieces a lane of a row that goes to a wave (0: none do) or to a
// block (-1: none do; 0: any number)
// Two pieces: eight waves a SIMD, which the scalar registers of both loops would
// otherwise not leave room for (65536 rows of 2048: 82.4 us with seven).
template <bool F32, int WAVE, int BLOCK>
__global__ __launch_bounds__(kRowWaves * kWave, WAVE == 2 ? 8 : 1) void quant_rows_kernel(QuantArgs p, int few) {
    __shared__ uint32_t s_max[2][kRowWaves];
    const int tid = threadIdx.x;
    long long r0 = 0, r1 = p.cap;
    if (p.m_counts != nullptr) {
        const int j = blockIdx.y;
        r0 = (long long)j * p.cap_e;
        r1 = r0 + min(max(p.m_counts[j], 0), p.cap_e);
    } else if (p.offsets != nullptr) {
        r0 = min(max(p.offsets[0], 0), p.cap);
        r1 = min(max(p.offsets[p.E_loc], (int)r0), p.cap);
    }
    if (BLOCK >= 0 && (WAVE == 0 || r1 - r0 <= few)) {
        // rows take turns with the two sets of s_max: the barrier of the row between
        // two that share one parts their reads and writes
        int turn = 0;
        for (long long r = r0 + blockIdx.x; r < r1; r += gridDim.x, turn ^= 1)
            quant_row<F32, BLOCK < 0 ? 0 : BLOCK, kRowWaves>(p, (size_t)r, tid, s_max[turn]);
    } else if (WAVE > 0) {
        const int wave = blockIdx.x * kRowWaves + __builtin_amdgcn_readfirstlane(tid / kWave);
        for (long long r = r0 + wave; r < r1; r += (long long)gridDim.x * kRowWaves)
            quant_row<F32, WAVE, 1>(p, (size_t)r, tid % kWave, nullptr);
    }
}

template <bool F32>
hipError_t launch_dispatch_any(const SegTable& seg, int B, int H, const int32_t* row_of, int K, uint8_t* xd,
                               float* xd_scales, int cap, hipStream_t stream) {
    // a batch that leaves CUs with room gets wider blocks (128 tokens of 7168: 5.7 us
    // with seven waves a token, 7.0 with four; 3684 tokens the other way: 20.6, 18.9)
    const int np = H / 16, waves = (np + kWave - 1) / kWave, most = B < 2 * device_cu_count() ? kTokThreads / kWave : 4;
    const dim3 grid(B), block(kWave * (waves < most ? waves : most));
    const int per = (np + (int)block.x - 1) / (int)block.x;
    if (per <= 1)
        hipLaunchKernelGGL((dispatch_i8_kernel<F32, 1>), grid, block, 0, stream, seg, H, row_of, K, cap, xd, xd_scales);
    else if (per <= 2)
        hipLaunchKernelGGL((dispatch_i8_kernel<F32, 2>), grid, block, 0, stream, seg, H, row_of, K, cap, xd, xd_scales);
    else if (per <= 4)
        hipLaunchKernelGGL((dispatch_i8_kernel<F32, 4>), grid, block, 0, stream, seg, H, row_of, K, cap, xd, xd_scales);
    else
        hipLaunchKernelGGL((dispatch_i8_kernel<F32, 0>), grid, block, 0, stream, seg, H, row_of, K, cap, xd, xd_scales);
    return hipGetLastError();
}

// few_per_cu: rows per CU up to which a row goes to a block
template <bool F32, int WAVE, int BLOCK>
hipError_t launch_quant_as(const QuantArgs& a, int few_per_cu, hipStream_t stream) {
    constexpr int kRows = BLOCK < 0 ? kRowWaves : 1;              // rows of a block at a time
    const int cus = device_cu_count(), most = cus * 8;
    int few = cus * few_per_cu;
    dim3 grid, block(kRowWaves * kWave);
    if (a.m_counts != nullptr) {
        few = (few + a.E_loc - 1) / a.E_loc;
        // two rows at least when a block of rows is full: decode fills few of them, and
        // workgroups with nothing to do cost more than the loop
        const int share = (most / 2 + a.E_loc - 1) / a.E_loc, need = (a.cap_e + 2 * kRows - 1) / (2 * kRows);
        grid = dim3(share < need ? share : need, a.E_loc);
    } else {
        const int need = (a.cap + kRows - 1) / kRows;
        grid = dim3(need < most ? need : most);
    }
    hipLaunchKernelGGL((quant_rows_kernel<F32, WAVE, BLOCK>), grid, block, 0, stream, a, few);
    return hipGetLastError();
}

template <bool F32>
hipError_t launch_quant_any(const QuantArgs& a, hipStream_t stream) {
    const int per = (a.cols / 16 + kWave - 1) / kWave;            // pieces a lane of a wave
    if (per <= 1) return launch_quant_as<F32, 1, -1>(a, 0, stream);
    if (per <= 2) return launch_quant_as<F32, 2, 1>(a, 8, stream);
    if (per <= 4) return launch_quant_as<F32, 4, 1>(a, 16, stream);
    if (per <= 8) return launch_quant_as<F32, 0, 2>(a, 0, stream);
    if (per <= 16) return launch_quant_as<F32, 0, 4>(a, 0, stream);
    if (per <= 32) return launch_quant_as<F32, 0, 8>(a, 0, stream);
    return launch_quant_as<F32, 0, 0>(a, 0, stream);
}

}  // namespace

hipError_t launch_dispatch_i8(const SegTable& seg, int B, int H, bool f32, const int32_t* row_of, int K, void* xd,
                              float* xd_scales, int cap, hipStream_t stream) {
    uint8_t* q = static_cast<uint8_t*>(xd);
    return launch_in_parts(B, [&](size_t b0, int n) {
        const SegTable part = seg.from(b0);
        const int32_t* rows = row_of + b0 * K;
        return f32 ? launch_dispatch_any<true>(part, n, H, rows, K, q, xd_scales, cap, stream)
                   : launch_dispatch_any<false>(part, n, H, rows, K, q, xd_scales, cap, stream);
    });
}

hipError_t launch_quant_rows(const QuantArgs& a, bool f32, hipStream_t stream) {
    if (a.cap == 0) return hipSuccess;
    return f32 ? launch_quant_any<true>(a, stream) : launch_quant_any<false>(a, stream);
}

}  // namespace moeep
