// The training step's grouped products in fp32 (the toy EP layer): gate/up with
// 8-bit checkpoints, input gradients, weight gradients.
//
// Sizes are small, so these are FMA kernels with LDS tiles on a persistent grid.
// Every sum runs in ascending order of its contraction index, so a result does
// not depend on the tile it falls into.
#include "ckpt_common.hpp"
#include "grouped_tiles.hpp"

namespace moeep {
namespace {

constexpr int kThreads = 256;
constexpr int kK = 16;                       // contraction steps of a chunk

template <typename T>
__device__ __forceinline__ float value(const T* p, size_t i) {
    if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)p[i] << 16);
    else return p[i];
}
template <typename T>
__device__ __forceinline__ void put(void* p, size_t i, float v) {
    if constexpr (sizeof(T) == 2) static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16_bits(v);
    else static_cast<float*>(p)[i] = v;
}

// ---- gate/up with checkpoints: 32 rows x 128 columns (one checkpoint block) of
// both products.  Thread (tx, ty) owns rows ty + 8 i and columns tx + 32 j, so the
// amax of a row's block is over 32 consecutive lanes.
constexpr int kRows = 32, kCols = 128;

template <typename T>
__global__ __launch_bounds__(kThreads) void gate_up_ckpt_kernel(FfnArgs p) {
    __shared__ float sA[kRows][kK + 1], sG[kCols][kK + 1], sU[kCols][kK + 1];
    __shared__ int s_pre[kMaxExperts + 1];
    __shared__ int s_tmp[kThreads / kWave];
    const int tid = threadIdx.x, tx = tid % 32, ty = tid / 32;
    const int Kdim = p.Kdim, N = p.N, ldw = p.ldw, nb = (N + kCkptBlock - 1) / kCkptBlock;
    build_tile_prefix<kThreads, kRows>(p, s_pre, s_tmp);
    const int n_tiles = (N + kCols - 1) / kCols, total = n_tiles * s_pre[p.E_loc];
    const T* A = static_cast<const T*>(p.a);
    for (int tau = blockIdx.x; tau < total; tau += gridDim.x) {
        const TileCoord tc = decode_tile<kRows>(tau, n_tiles, s_pre, p);
        const int col0 = tc.nt * kCols;
        const T* wg = static_cast<const T*>(p.w0) + (size_t)tc.j * N * ldw;
        const T* wu = static_cast<const T*>(p.w1) + (size_t)tc.j * N * ldw;
        float g[4][4] = {}, u[4][4] = {};
        for (int k0 = 0; k0 < Kdim; k0 += kK) {
            __syncthreads();
            for (int i = tid; i < kRows * kK; i += kThreads) {
                const int r = i / kK, k = i % kK;
                sA[r][k] = r < tc.nvalid && k0 + k < Kdim ? value(A, (size_t)(tc.row0 + r) * Kdim + k0 + k) : 0.0f;
            }
            for (int i = tid; i < kCols * kK; i += kThreads) {
                const int c = i / kK, k = i % kK;
                const bool in = col0 + c < N && k0 + k < Kdim;
                const size_t at = (size_t)(col0 + c) * ldw + k0 + k;
                sG[c][k] = in ? value(wg, at) : 0.0f;
                sU[c][k] = in ? value(wu, at) : 0.0f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kK; ++k) {
                float a[4], wgv[4], wuv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = sA[ty + 8 * i][k];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    wgv[j] = sG[tx + 32 * j][k];
                    wuv[j] = sU[tx + 32 * j][k];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        g[i][j] = fmaf(a[i], wgv[j], g[i][j]);
                        u[i][j] = fmaf(a[i], wuv[j], u[i][j]);
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 8 * i;
            uint32_t mg = 0, mu = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {       // columns past N hold zeros
                mg = max(mg, __float_as_uint(g[i][j]) & 0x7fffffffu);
                mu = max(mu, __float_as_uint(u[i][j]) & 0x7fffffffu);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                mg = max(mg, (uint32_t)__shfl_xor((int)mg, d, kWave));
                mu = max(mu, (uint32_t)__shfl_xor((int)mu, d, kWave));
            }
            if (r >= tc.nvalid) continue;
            const float gs = ckpt_scale(mg), us = ckpt_scale(mu), grs = ckpt_recip(gs), urs = ckpt_recip(us);
            const size_t row = (size_t)(tc.row0 + r);
            if (tx == 0) {
                p.gate_s[row * nb + tc.nt] = gs;
                p.up_s[row * nb + tc.nt] = us;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = col0 + tx + 32 * j;
                if (c >= N) continue;
                p.gate_q[row * N + c] = gs == gs ? (int8_t)ckpt_code(g[i][j], grs) : (int8_t)0;
                p.up_q[row * N + c] = us == us ? (int8_t)ckpt_code(u[i][j], urs) : (int8_t)0;
                put<T>(p.out, row * N + c, g[i][j] / (1.0f + expf(-g[i][j])) * u[i][j]);
            }
        }
    }
}

// ---- 64 x 64 tiles of the gradients: thread (tx, ty) owns rows ty + 16 i and
// columns tx + 16 j
constexpr int kTile = 64;

struct Tile {
    float a[kK][kTile + 1], b[kK][kTile + 1];

    __device__ __forceinline__ void multiply(float (&acc)[4][4], int tx, int ty) const {
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            float av[4], bv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                av[i] = a[k][ty + 16 * i];
                bv[i] = b[k][tx + 16 * i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
        }
    }
};

// the operand row that the expert row r reads, -1 if src_of names none of src_rows
__device__ __forceinline__ int gathered(const int32_t* src_of, int per, int src_rows, int r) {
    if (src_of == nullptr) return r;
    const int s = src_of[r];
    const int t = s < 0 ? -1 : s / per;
    return t < src_rows ? t : -1;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dgrad_kernel(FfnArgs p) {
    __shared__ Tile s;
    __shared__ int s_row[kTile];
    __shared__ int s_pre[kMaxExperts + 1];
    __shared__ int s_tmp[kThreads / kWave];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int Kdim = p.Kdim, N = p.N, ldw = p.ldw;
    build_tile_prefix<kThreads, kTile>(p, s_pre, s_tmp);
    const int n_tiles = (N + kTile - 1) / kTile, total = n_tiles * s_pre[p.E_loc];
    for (int tau = blockIdx.x; tau < total; tau += gridDim.x) {
        const TileCoord tc = decode_tile<kTile>(tau, n_tiles, s_pre, p);
        const int col0 = tc.nt * kTile;
        __syncthreads();
        if (tid < kTile) s_row[tid] = tid < tc.nvalid ? gathered(p.src_of, p.per, p.src_rows, tc.row0 + tid) : -1;
        float acc[4][4] = {};
        for (int q = 0; q < 2; ++q) {
            const T* A = static_cast<const T*>(q == 0 ? p.a : p.a2);
            if (A == nullptr) break;
            const T* W = static_cast<const T*>(q == 0 ? p.w0 : p.w1) + (size_t)tc.j * Kdim * ldw;
            for (int k0 = 0; k0 < Kdim; k0 += kK) {
                __syncthreads();
                for (int i = tid; i < kTile * kK; i += kThreads) {
                    const int r = i / kK, k = i % kK, row = s_row[r];
                    s.a[k][r] = row >= 0 && k0 + k < Kdim ? value(A, (size_t)row * Kdim + k0 + k) : 0.0f;
                }
                for (int i = tid; i < kTile * kK; i += kThreads) {
                    const int k = i / kTile, c = i % kTile;
                    s.b[k][c] = k0 + k < Kdim && col0 + c < N ? value(W, (size_t)(k0 + k) * ldw + col0 + c) : 0.0f;
                }
                __syncthreads();
                s.multiply(acc, tx, ty);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ty + 16 * i, c = col0 + tx + 16 * j;
                if (r < tc.nvalid && c < N) put<T>(p.out, (size_t)(tc.row0 + r) * N + c, acc[i][j]);
            }
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void wgrad_kernel(WgradArgs p, long long tiles) {
    __shared__ Tile s;
    __shared__ int s_dy[kK], s_x[kK];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int N = p.N, M = p.M, tm = (M + kTile - 1) / kTile, tn = (N + kTile - 1) / kTile;
    const int nb = (M + kCkptBlock - 1) / kCkptBlock;
    for (long long tau = blockIdx.x; tau < tiles; tau += gridDim.x) {
        long long rest = tau;
        const int m0 = (int)(rest % tm) * kTile;
        rest /= tm;
        const int n0 = (int)(rest % tn) * kTile;
        rest /= tn;
        const int pairs = p.dy[1] != nullptr ? 2 : 1, q = (int)(rest % pairs), j = (int)(rest / pairs);
        const T* dy = static_cast<const T*>(p.dy[q]);
        const int r0 = clampi(p.offsets[j], 0, p.cap), r1 = clampi(p.offsets[j + 1], r0, p.cap);
        float acc[4][4] = {};
        for (int r = r0; r < r1; r += kK) {
            __syncthreads();
            if (tid < kK) {
                const int g = r + tid < r1 ? gathered(p.src_of, p.per, p.src_rows, r + tid) : -1;
                const int own = r + tid < r1 ? r + tid : -1;
                s_dy[tid] = p.gather_dy ? g : own;
                s_x[tid] = p.gather_x ? g : own;
            }
            __syncthreads();
            for (int i = tid; i < kTile * kK; i += kThreads) {
                const int k = i / kTile, c = i % kTile, a = s_dy[k], b = s_x[k];
                s.a[k][c] = a >= 0 && n0 + c < N ? value(dy, (size_t)a * N + n0 + c) : 0.0f;
                float x = 0.0f;
                if (b >= 0 && m0 + c < M) {
                    const size_t at = (size_t)b * M + m0 + c;
                    if (p.x_scales != nullptr)
                        x = (float)static_cast<const int8_t*>(p.x)[at] * p.x_scales[(size_t)b * nb + (m0 + c) / kCkptBlock];
                    else x = value(static_cast<const T*>(p.x), at);
                }
                s.b[k][c] = x;
            }
            __syncthreads();
            s.multiply(acc, tx, ty);
        }
        const size_t w0 = (size_t)j * N * M;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                const int n = n0 + ty + 16 * i, m = m0 + tx + 16 * jj;
                if (n >= N || m >= M) continue;
                const size_t at = w0 + (size_t)n * M + m;
                float v = acc[i][jj];
                if (p.base[q] != nullptr)
                    v += p.dw_f32 ? static_cast<const float*>(p.base[q])[at]
                                  : value(static_cast<const uint16_t*>(p.base[q]), at);
                if (p.dw_f32) put<float>(p.dw[q], at, v);
                else put<uint16_t>(p.dw[q], at, v);
            }
    }
}

template <typename T>
hipError_t wgrad(const WgradArgs& a, hipStream_t stream) {
    const long long tiles = (long long)a.E_loc * (a.dy[1] != nullptr ? 2 : 1) * ((a.N + kTile - 1) / kTile) *
                            ((a.M + kTile - 1) / kTile);
    const int most = device_cu_count() * 8;
    hipLaunchKernelGGL(wgrad_kernel<T>, dim3(tiles < most ? (int)tiles : most), dim3(kThreads), 0, stream, a, tiles);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ffn_ckpt_f32(const FfnArgs& a, hipStream_t stream) {
    static int per_cu = 0;
    return launch_persistent(gate_up_ckpt_kernel<float>, kThreads, a, stream, &per_cu);
}
hipError_t launch_dgrad_f32(const FfnArgs& a, hipStream_t stream) {
    static int per_cu = 0;
    return launch_persistent(dgrad_kernel<float>, kThreads, a, stream, &per_cu);
}
hipError_t launch_wgrad_f32(const WgradArgs& a, hipStream_t stream) { return wgrad<float>(a, stream); }

}  // namespace moeep
