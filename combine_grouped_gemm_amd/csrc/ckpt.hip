// 8-bit checkpoints of rows (the format: ckpt_common.hpp), and SwiGLU's
// backward pass from checkpoints of gate and up.
//
// All three kernels move data and little else: 8 consecutive columns a lane, so
// that a block of 128 is a DPP row of 16 lanes and its amax four lane moves.
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
// cancel.  A wave takes `chunk` consecutive slots: it reads their rows at once,
// writes zeros for those without one, and walks the others.
template <bool F32>
__global__ __launch_bounds__(kWaves * kWave) void swiglu_backward_kernel(SwigluBwdArgs p, int chunk) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int nb = (p.I + kCkptBlock - 1) / kCkptBlock;
    constexpr int kSize = F32 ? 4 : 2;
    for (long long s0 = ((long long)blockIdx.x * kWaves + wave) * chunk; s0 < p.slots;
         s0 += (long long)gridDim.x * kWaves * chunk) {
        int my = -1;
        float my_w = 0.0f;
        const bool mine = lane < chunk && s0 + lane < p.slots;
        if (mine) {
            const int r = p.row_of[s0 + lane];
            my = r >= 0 && r < p.cap ? r : -1;
            my_w = p.topk_w[s0 + lane];
        }
        uint64_t todo = ballot64(my >= 0);
        float my_dw = 0.0f;
        while (todo != 0) {
            const int k = __builtin_ctzll(todo);
            todo &= todo - 1;
            const int r = __builtin_amdgcn_readlane(my, k);
            const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_w), k));
            const size_t at = (size_t)r * p.I, sat = (size_t)r * nb;
            const char* dh_row = static_cast<const char*>(p.dh) + at * kSize;
            float sum = 0.0f;
#pragma unroll 2
            for (int c = lane * 8; c < p.I; c += 512) {
                Eight<F32> d;
                d.load(dh_row + (size_t)c * kSize);
                const uint2 gq = *reinterpret_cast<const uint2*>(p.gate_q + at + c);
                const uint2 uq = *reinterpret_cast<const uint2*>(p.up_q + at + c);
                float g[8], u[8], dh[8], dg[8], du[8], hw[8];
                code_values(gq, p.gate_s[sat + c / kCkptBlock], g);
                code_values(uq, p.up_s[sat + c / kCkptBlock], u);
                d.values(dh);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // e^-g overflows for g < -88: sg = 0, 1 - sg = 1
                    const float e = F32 ? expf(-g[i]) : __expf(-g[i]);
                    const float sg = F32 ? 1.0f / (1.0f + e) : __builtin_amdgcn_rcpf(1.0f + e);
                    const float rest = e < 3e38f ? e * sg : 1.0f;                // 1 - sg
                    const float act = g[i] * sg, wd = w * dh[i], h = act * u[i];
                    dg[i] = wd * u[i] * fmaf(act, rest, sg);
                    du[i] = wd * act;
                    hw[i] = w * h;
                    sum = fmaf(dh[i], h, sum);
                }
                Eight<F32>::store(static_cast<char*>(p.dgate) + (at + c) * kSize, dg);
                Eight<F32>::store(static_cast<char*>(p.dup) + (at + c) * kSize, du);
                Eight<F32>::store(static_cast<char*>(p.hw) + (at + c) * kSize, hw);
            }
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, kWave);
            if (lane == k) my_dw = sum;
        }
        if (mine) p.dtopk_w[s0 + lane] = my_dw;
    }
}

dim3 row_grid(const CkptArgs& a) {
    const int pieces = (a.cols + kPieceCols - 1) / kPieceCols;
    const int need = (a.cap + kWaves - 1) / kWaves, most = (device_cu_count() * 8 + pieces - 1) / pieces;
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
    const int most = device_cu_count() * 8;
    // one slot a wave while there are few, up to 16 when a launch has many
    int chunk = 1;
    while (chunk < 16 && a.slots > (long long)most * kWaves * chunk) chunk *= 2;
    const long long need = (a.slots + (long long)kWaves * chunk - 1) / ((long long)kWaves * chunk);
    const dim3 grid(need < most ? (int)need : most), block(kWaves * kWave);
    if (f32) hipLaunchKernelGGL(swiglu_backward_kernel<true>, grid, block, 0, stream, a, chunk);
    else hipLaunchKernelGGL(swiglu_backward_kernel<false>, grid, block, 0, stream, a, chunk);
    return hipGetLastError();
}

}  // namespace moeep
