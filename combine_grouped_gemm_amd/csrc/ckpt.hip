// 8-bit checkpoints of rows (the format: ckpt_common.hpp), and SwiGLU's
// backward pass from checkpoints of gate and up.
//
// All three kernels move data and little else: 8 consecutive columns a lane, so
// that a block of 128 is a DPP row of 16 lanes and its amax four lane moves.  A row goes in
// pieces of 2048 columns, whose loads are all in flight at once.  8192 rows of 7168 bf16
// columns: 44 us to pack (4.1 TB/s; 31 where x lies in the Infinity Cache), 28 back (6.4, the codes
// still in that cache); a copy 4.9 TB/s.
#include "ckpt_common.hpp"
#include "launch.hpp"

namespace moeep {
namespace {

constexpr int kWaves = 4;                    // waves of a block
constexpr int kPiece = 4;                    // 512-column steps of a wave's piece of a row
constexpr int kPieceCols = kPiece * 512;

// 8 consecutive values of a row, as they are in memory: 16 bytes of bf16 or 32 of fp32.
template <bool F32>
struct Eight {
    uint4 v[F32 ? 2 : 1];

    __device__ __forceinline__ void load(const void* p) {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = static_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void values(float (&f)[8]) const {
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[i * 4] = __uint_as_float(v[i].x);
                f[i * 4 + 1] = __uint_as_float(v[i].y);
                f[i * 4 + 2] = __uint_as_float(v[i].z);
                f[i * 4 + 3] = __uint_as_float(v[i].w);
            }
        } else {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f[k * 2] = bf16_lo(w[k]);
                f[k * 2 + 1] = bf16_hi(w[k]);
            }
        }
    }
    // rounded to bf16 to nearest even; fp32 as they are
    static __device__ __forceinline__ void store(void* p, const float (&f)[8]) {
        uint4* d = static_cast<uint4*>(p);
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                d[i] = make_uint4(__float_as_uint(f[i * 4]), __float_as_uint(f[i * 4 + 1]), __float_as_uint(f[i * 4 + 2]),
                                  __float_as_uint(f[i * 4 + 3]));
        } else {
            d[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                              pack_bf16x2(f[6], f[7]));
        }
    }
};

__device__ __forceinline__ void code_values(uint2 q, float s, float (&f)[8]) {
    f[0] = code_value<0>(q.x) * s;
    f[1] = code_value<1>(q.x) * s;
    f[2] = code_value<2>(q.x) * s;
    f[3] = code_value<3>(q.x) * s;
    f[4] = code_value<0>(q.y) * s;
    f[5] = code_value<1>(q.y) * s;
    f[6] = code_value<2>(q.y) * s;
    f[7] = code_value<3>(q.y) * s;
}

// the rows a call works on: all, or those of the contiguous layout's experts
__device__ __forceinline__ void valid_rows(const CkptArgs& p, long long& r0, long long& r1) {
    r0 = 0;
    r1 = p.cap;
    if (p.offsets != nullptr) {
        r0 = min(max(p.offsets[0], 0), p.cap);
        r1 = min(max(p.offsets[p.E_loc], (int)r0), p.cap);
    }
}

// blockIdx.y: the piece of a row; a wave takes every (4 gridDim.x)-th row
template <bool F32>
__global__ __launch_bounds__(kWaves * kWave) void checkpoint_rows_kernel(CkptArgs p) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int nb = (p.cols + kCkptBlock - 1) / kCkptBlock, c0 = blockIdx.y * kPieceCols + lane * 8;
    constexpr int kSize = F32 ? 4 : 2;
    long long r0, r1;
    valid_rows(p, r0, r1);
    for (long long r = r0 + (long long)blockIdx.x * kWaves + wave; r < r1; r += (long long)gridDim.x * kWaves) {
        const char* row = static_cast<const char*>(p.x) + (size_t)r * p.cols * kSize;
        Eight<F32> v[kPiece];
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
            const int c = c0 + i * 512;
            if (c < p.cols) v[i].load(row + (size_t)c * kSize);
            else v[i].zero();
        }
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
            const int c = c0 + i * 512;
            float f[8];
            v[i].values(f);
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t u = __float_as_uint(f[k]) & 0x7fffffffu;
                m = u > m ? u : m;
            }
            const float s = ckpt_scale(row16_max_u32(m)), rs = ckpt_recip(s);
            uint32_t t[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) t[k] = ckpt_code(f[k], rs);
            uint2 q = make_uint2(pack_low_bytes(t[0], t[1], t[2], t[3]), pack_low_bytes(t[4], t[5], t[6], t[7]));
            if (s != s) q = make_uint2(0, 0);
            if (c < p.cols) {
                *reinterpret_cast<uint2*>(p.q + (size_t)r * p.cols + c) = q;
                if (lane % 16 == 0) p.scales[(size_t)r * nb + c / kCkptBlock] = s;
            }
        }
    }
}

template <bool F32>
__global__ __launch_bounds__(kWaves * kWave) void checkpoint_values_kernel(CkptArgs p) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int nb = (p.cols + kCkptBlock - 1) / kCkptBlock, c0 = blockIdx.y * kPieceCols + lane * 8;
    constexpr int kSize = F32 ? 4 : 2;
    long long r0, r1;
    valid_rows(p, r0, r1);
    for (long long r = r0 + (long long)blockIdx.x * kWaves + wave; r < r1; r += (long long)gridDim.x * kWaves) {
        char* row = static_cast<char*>(p.x) + (size_t)r * p.cols * kSize;
        uint2 q[kPiece];
        float s[kPiece];
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
            const int c = c0 + i * 512;
            if (c < p.cols) {
                q[i] = *reinterpret_cast<const uint2*>(p.q + (size_t)r * p.cols + c);
                s[i] = p.scales[(size_t)r * nb + c / kCkptBlock];
            }
        }
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
            const int c = c0 + i * 512;
            if (c < p.cols) {
                float f[8];
                code_values(q[i], s[i], f);
                Eight<F32>::store(row + (size_t)c * kSize, f);
            }
        }
    }
}

// SwiGLU backwards, for the row of every slot:
//   sg = 1 / (1 + e^-g), h = g sg u
//   dgate = w dh u sg (1 + g (1 - sg)), dup = w dh g sg, hw = w h, dw = <dh, h>
// dh is the gradient of the unweighted expert output's h, so <dh, h> is the
// gradient of the slot's weight w.  1 - sg comes from e^-g itself and does not
// cancel.
//
// A block takes `per` consecutive slots (4 to 32).  Its first wave reads their rows, writes the
// zeros of those that have none and lists the others in LDS; the waves share the list a row
// each.  So ranks that hold an eighth of the slots keep their waves busy alike (8192 of
// 65536 slots, 2048 columns: a wave that walked its own 8 slots 54 us, this 44, 3.8 TB/s), and a
// wave has all loads of 2048 columns in flight.
constexpr int kSlots = 32;

template <bool F32>
__global__ __launch_bounds__(kWaves * kWave, 4) void swiglu_backward_kernel(SwigluBwdArgs p, int per) {
    __shared__ int s_row[kSlots], s_slot[kSlots], s_n;
    __shared__ float s_w[kSlots];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int nb = (p.I + kCkptBlock - 1) / kCkptBlock;
    constexpr int kSize = F32 ? 4 : 2;
    for (long long s0 = (long long)blockIdx.x * per; s0 < p.slots; s0 += (long long)gridDim.x * per) {
        __syncthreads();                             // the list before is used up
        if (tid < kWave) {
            int r = -1;
            const bool mine = lane < per && s0 + lane < p.slots;
            if (mine) {
                r = p.row_of[s0 + lane];
                if (r < 0 || r >= p.cap) {
                    r = -1;
                    p.dtopk_w[s0 + lane] = 0.0f;
                }
            }
            const uint64_t local = ballot64(r >= 0);
            if (r >= 0) {
                const int at = popc64(local & lanemask_lt());
                s_row[at] = r;
                s_slot[at] = lane;
                s_w[at] = p.topk_w[s0 + lane];
            }
            if (lane == 0) s_n = popc64(local);
        }
        __syncthreads();
        const int n = s_n;
        for (int i = wave; i < n; i += kWaves) {
            const int r = __builtin_amdgcn_readfirstlane(s_row[i]);
            const float w = s_w[i];
            const size_t at = (size_t)r * p.I, sat = (size_t)r * nb;
            const char* dh_row = static_cast<const char*>(p.dh) + at * kSize;
            float sum = 0.0f;
            for (int c0 = 0; c0 < p.I; c0 += kPieceCols) {
                Eight<F32> d[kPiece];
                uint2 gq[kPiece], uq[kPiece];
                float gs[kPiece], us[kPiece];
#pragma unroll
                for (int k = 0; k < kPiece; ++k) {
                    const int c = c0 + k * 512 + lane * 8;
                    if (c < p.I) {
                        d[k].load(dh_row + (size_t)c * kSize);
                        gq[k] = *reinterpret_cast<const uint2*>(p.gate_q + at + c);
                        uq[k] = *reinterpret_cast<const uint2*>(p.up_q + at + c);
                        gs[k] = p.gate_s[sat + c / kCkptBlock];
                        us[k] = p.up_s[sat + c / kCkptBlock];
                    }
                }
#pragma unroll
                for (int k = 0; k < kPiece; ++k) {
                    const int c = c0 + k * 512 + lane * 8;
                    if (c >= p.I) continue;
                    float g[8], u[8], dh[8], dg[8], du[8], hw[8];
                    code_values(gq[k], gs[k], g);
                    code_values(uq[k], us[k], u);
                    d[k].values(dh);
#pragma unroll
                    for (int e8 = 0; e8 < 8; ++e8) {
                        // e^-g overflows for g < -88: sg = 0, 1 - sg = 1
                        const float e = F32 ? expf(-g[e8]) : __expf(-g[e8]);
                        const float sg = F32 ? 1.0f / (1.0f + e) : __builtin_amdgcn_rcpf(1.0f + e);
                        const float rest = e < 3e38f ? e * sg : 1.0f;                // 1 - sg
                        const float act = g[e8] * sg, wd = w * dh[e8], h = act * u[e8];
                        dg[e8] = wd * u[e8] * fmaf(act, rest, sg);
                        du[e8] = wd * act;
                        hw[e8] = w * h;
                        sum = fmaf(dh[e8], h, sum);
                    }
                    Eight<F32>::store(static_cast<char*>(p.dgate) + (at + c) * kSize, dg);
                    Eight<F32>::store(static_cast<char*>(p.dup) + (at + c) * kSize, du);
                    Eight<F32>::store(static_cast<char*>(p.hw) + (at + c) * kSize, hw);
                }
            }
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, kWave);
            if (lane == 0) p.dtopk_w[s0 + s_slot[i]] = sum;
        }
    }
}

dim3 row_grid(const CkptArgs& a) {
    const int pieces = (a.cols + kPieceCols - 1) / kPieceCols;
    const int need = a.cap / kWaves + (a.cap % kWaves != 0), most = (device_cu_count() * 8 + pieces - 1) / pieces;
    return dim3(need < most ? need : most, pieces);
}

}  // namespace

hipError_t launch_checkpoint_rows(const CkptArgs& a, bool f32, hipStream_t stream) {
    if (a.cap == 0) return hipSuccess;
    const dim3 block(kWaves * kWave);
    if (f32) hipLaunchKernelGGL(checkpoint_rows_kernel<true>, row_grid(a), block, 0, stream, a);
    else hipLaunchKernelGGL(checkpoint_rows_kernel<false>, row_grid(a), block, 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_checkpoint_values(const CkptArgs& a, bool f32, hipStream_t stream) {
    if (a.cap == 0) return hipSuccess;
    const dim3 block(kWaves * kWave);
    if (f32) hipLaunchKernelGGL(checkpoint_values_kernel<true>, row_grid(a), block, 0, stream, a);
    else hipLaunchKernelGGL(checkpoint_values_kernel<false>, row_grid(a), block, 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_swiglu_backward(const SwigluBwdArgs& a, bool f32, hipStream_t stream) {
    if (a.slots == 0) return hipSuccess;
    // a slot a wave while there are few; a list long enough to share once they fill the device
    const int most = device_cu_count() * 8;
    int per = kWaves;
    while (per < kSlots && a.slots > (long long)device_cu_count() * 4 * per) per *= 2;
    const long long need = (a.slots + per - 1) / per;
    const dim3 grid(need < most ? (int)need : most), block(kWaves * kWave);
    if (f32) hipLaunchKernelGGL(swiglu_backward_kernel<true>, grid, block, 0, stream, a, per);
    else hipLaunchKernelGGL(swiglu_backward_kernel<false>, grid, block, 0, stream, a, per);
    return hipGetLastError();
}

}  // namespace moeep
