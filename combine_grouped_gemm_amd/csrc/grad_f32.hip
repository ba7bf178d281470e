// The training step's grouped products in fp32 (the toy EP layer): gate/up with
// 8-bit checkpoints, input gradients, weight gradients.
//
// Sizes are small, so small tiles: 64 x 64 of a gradient, 32 x 32 where that leaves CUs
// without one, 32 rows x 128 columns of both gate and up (a checkpoint block), four waves,
// 32-deep contraction chunks that go through registers into LDS while the chunk before is
// multiplied.  The products are v_mfma_f32_16x16x4_f32: fp32 operands, fp32 sums; lane l feeds row (column) l % 16 with
// k = l / 16 and receives rows 4 (l / 16) + e, column l % 16.
//
// Operands lie in LDS as they do in memory.  Contraction along the row ([r][k], pitch 36):
// the 16 rows x 4 k of an operand read fall into 64 different banks (36 r mod 64 takes
// every multiple of 4).  Contraction over rows ([k][c], pitch 80 or 48): 4 rows of 16
// columns, 16 banks apart.
//
// Bound by latency at the toy layer's sizes, by LDS reads and few blocks a CU beyond: 8
// experts, 1024 x 1024, gate/up of 128 rows each 58 us (74 TFLOP/s), a pair's input gradient of
// 512 rows 160 us (107); 16 experts of 256 rows, 512 x 1024, weight gradients 52 us (82).  Where
// 32 x 32 tiles are taken, beside 64 x 64 ones on one card: 4 experts of 10 rows, a pair at 1024 x
// 1024, 34 us and 61; 256 x 256 weight gradients of 512 rows 16 us and 29.
#include "ckpt_common.hpp"
#include "grouped_tiles.hpp"

namespace moeep {
namespace {

constexpr int kThreads = 256;
constexpr int kK = 32;                       // contraction steps of a chunk
constexpr int kPitchK = 36;                  // floats, [r][k]
template <int T>                             // floats, [k][T columns]
constexpr int kPitchC = T == 64 ? 80 : 48;

__device__ __forceinline__ floatx4 mma(float a, float b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// the operand row that the expert row r reads, -1 if src_of names none of src_rows
__device__ __forceinline__ int gathered(const int32_t* src_of, int per, int src_rows, int r) {
    if (src_of == nullptr) return r;
    const int s = src_of[r];
    const int t = s < 0 ? -1 : s / per;
    return t < src_rows ? t : -1;
}

__device__ __forceinline__ float4 zero4() { return make_float4(0.0f, 0.0f, 0.0f, 0.0f); }

// ---- gate/up with checkpoints: wave w has columns 32 w .. + 31 of both products
constexpr int kRows = 32, kCols = 128;

__global__ __launch_bounds__(kThreads) void gate_up_ckpt_kernel(FfnArgs p) {
    __shared__ __align__(16) float sA[kRows * kPitchK], sG[kCols * kPitchK], sU[kCols * kPitchK];
    __shared__ uint2 s_max[kRows][4];
    __shared__ int s_pre[kMaxExperts + 1];
    __shared__ int s_tmp[kThreads / kWave];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, r16 = lane & 15, g4 = lane >> 4;
    const int Kdim = p.Kdim, N = p.N, ldw = p.ldw, nb = (N + kCkptBlock - 1) / kCkptBlock;
    build_tile_prefix<kThreads, kRows>(p, s_pre, s_tmp);
    const int n_tiles = (N + kCols - 1) / kCols, total = n_tiles * s_pre[p.E_loc];
    const float* A = static_cast<const float*>(p.a);
    float* Out = static_cast<float*>(p.out);
    const int lr = tid / 8, lk = (tid % 8) * 4;              // row and first k of a thread's pieces
    for (int tau = blockIdx.x; tau < total; tau += gridDim.x) {
        const TileCoord tc = decode_tile<kRows>(tau, n_tiles, s_pre, p);
        const int col0 = tc.nt * kCols;
        const float* wg = static_cast<const float*>(p.w0) + (size_t)tc.j * N * ldw;
        const float* wu = static_cast<const float*>(p.w1) + (size_t)tc.j * N * ldw;
        float4 ra, rg[4], ru[4];
        auto load = [&](int k0) {
            const int k = k0 + lk;
            ra = lr < tc.nvalid && k < Kdim ? *reinterpret_cast<const float4*>(A + (size_t)(tc.row0 + lr) * Kdim + k) : zero4();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = col0 + i * 32 + lr;
                const bool in = c < N && k < Kdim;
                rg[i] = in ? *reinterpret_cast<const float4*>(wg + (size_t)c * ldw + k) : zero4();
                ru[i] = in ? *reinterpret_cast<const float4*>(wu + (size_t)c * ldw + k) : zero4();
            }
        };
        floatx4 g[2][2] = {}, u[2][2] = {};
        load(0);
        for (int k0 = 0; k0 < Kdim; k0 += kK) {
            __syncthreads();
            *reinterpret_cast<float4*>(sA + lr * kPitchK + lk) = ra;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                *reinterpret_cast<float4*>(sG + (i * 32 + lr) * kPitchK + lk) = rg[i];
                *reinterpret_cast<float4*>(sU + (i * 32 + lr) * kPitchK + lk) = ru[i];
            }
            __syncthreads();
            if (k0 + kK < Kdim) load(k0 + kK);
#pragma unroll
            for (int k = 0; k < kK; k += 4) {
                float a[2], b[2], c[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    a[i] = sA[(i * 16 + r16) * kPitchK + k + g4];
                    b[i] = sG[(wave * 32 + i * 16 + r16) * kPitchK + k + g4];
                    c[i] = sU[(wave * 32 + i * 16 + r16) * kPitchK + k + g4];
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        g[i][j] = mma(a[i], b[j], g[i][j]);
                        u[i][j] = mma(a[i], c[j], u[i][j]);
                    }
            }
        }
        // each row's largest magnitudes over the block's 128 columns (those past N hold zeros)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t mg = row16_max_u32(max(__float_as_uint(g[i][0][e]) & 0x7fffffffu,
                                                      __float_as_uint(g[i][1][e]) & 0x7fffffffu));
                const uint32_t mu = row16_max_u32(max(__float_as_uint(u[i][0][e]) & 0x7fffffffu,
                                                      __float_as_uint(u[i][1][e]) & 0x7fffffffu));
                if (r16 == 0) s_max[i * 16 + g4 * 4 + e][wave] = make_uint2(mg, mu);
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = i * 16 + g4 * 4 + e;
                if (r >= tc.nvalid) continue;
                uint2 m = s_max[r][0];
#pragma unroll
                for (int w = 1; w < 4; ++w) m = make_uint2(max(m.x, s_max[r][w].x), max(m.y, s_max[r][w].y));
                const float gs = ckpt_scale(m.x), us = ckpt_scale(m.y), grs = ckpt_recip(gs), urs = ckpt_recip(us);
                const size_t row = (size_t)(tc.row0 + r);
                if (wave == 0 && r16 == 0) {
                    p.gate_s[row * nb + tc.nt] = gs;
                    p.up_s[row * nb + tc.nt] = us;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = col0 + wave * 32 + j * 16 + r16;
                    if (c >= N) continue;
                    const float gv = g[i][j][e], uv = u[i][j][e];
                    p.gate_q[row * N + c] = gs == gs ? (int8_t)ckpt_code(gv, grs) : (int8_t)0;
                    p.up_q[row * N + c] = us == us ? (int8_t)ckpt_code(uv, urs) : (int8_t)0;
                    Out[row * N + c] = gv / (1.0f + expf(-gv)) * uv;
                }
            }
    }
}

// ---- gradients: wave (wr, wc) of 2 x 2 has a quarter of a T x T tile
template <int T>
__global__ __launch_bounds__(kThreads) void dgrad_kernel(FfnArgs p) {
    constexpr int F = T / 32, PC = kPitchC<T>, Q = T / 4;        // fragments a side, 16-byte pieces of a row
    __shared__ __align__(16) float sA[T * kPitchK], sB[kK * PC];
    __shared__ int s_row[T];
    __shared__ int s_pre[kMaxExperts + 1];
    __shared__ int s_tmp[kThreads / kWave];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, r16 = lane & 15, g4 = lane >> 4;
    const int wr = wave / 2 * (T / 2), wc = wave % 2 * (T / 2);
    const int Kdim = p.Kdim, N = p.N, ldw = p.ldw;
    build_tile_prefix<kThreads, T>(p, s_pre, s_tmp);
    const int n_tiles = (N + T - 1) / T, total = n_tiles * s_pre[p.E_loc];
    float* Out = static_cast<float*>(p.out);
    for (int tau = blockIdx.x; tau < total; tau += gridDim.x) {
        const TileCoord tc = decode_tile<T>(tau, n_tiles, s_pre, p);
        const int col0 = tc.nt * T;
        __syncthreads();
        if (tid < T) s_row[tid] = tid < tc.nvalid ? gathered(p.src_of, p.per, p.src_rows, tc.row0 + tid) : -1;
        __syncthreads();
        floatx4 acc[F][F] = {};
        for (int q = 0; q < 2; ++q) {
            const float* A = static_cast<const float*>(q == 0 ? p.a : p.a2);
            if (A == nullptr) break;
            const float* W = static_cast<const float*>(q == 0 ? p.w0 : p.w1) + (size_t)tc.j * Kdim * ldw;
            float4 ra[F], rb[F];
            auto load = [&](int k0) {
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    const int row = s_row[i * 32 + tid / 8], k = k0 + (tid % 8) * 4;
                    ra[i] = row >= 0 && k < Kdim ? *reinterpret_cast<const float4*>(A + (size_t)row * Kdim + k) : zero4();
                    const int kb = k0 + i * (kThreads / Q) + tid / Q, c = col0 + (tid % Q) * 4;
                    rb[i] = kb < Kdim && c < N ? *reinterpret_cast<const float4*>(W + (size_t)kb * ldw + c) : zero4();
                }
            };
            load(0);
            for (int k0 = 0; k0 < Kdim; k0 += kK) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    *reinterpret_cast<float4*>(sA + (i * 32 + tid / 8) * kPitchK + (tid % 8) * 4) = ra[i];
                    *reinterpret_cast<float4*>(sB + (i * (kThreads / Q) + tid / Q) * PC + (tid % Q) * 4) = rb[i];
                }
                __syncthreads();
                if (k0 + kK < Kdim) load(k0 + kK);
#pragma unroll
                for (int k = 0; k < kK; k += 4) {
                    float a[F], b[F];
#pragma unroll
                    for (int i = 0; i < F; ++i) {
                        a[i] = sA[(wr + i * 16 + r16) * kPitchK + k + g4];
                        b[i] = sB[(k + g4) * PC + wc + i * 16 + r16];
                    }
#pragma unroll
                    for (int i = 0; i < F; ++i)
#pragma unroll
                        for (int j = 0; j < F; ++j) acc[i][j] = mma(a[i], b[j], acc[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = wr + i * 16 + g4 * 4 + e, c = col0 + wc + j * 16 + r16;
                    if (r < tc.nvalid && c < N) Out[(size_t)(tc.row0 + r) * N + c] = acc[i][j][e];
                }
    }
}

template <int T>
__global__ __launch_bounds__(kThreads) void wgrad_kernel(WgradArgs p, int tiles) {
    constexpr int F = T / 32, PC = kPitchC<T>, Q = T / 4;
    __shared__ __align__(16) float sY[kK * PC], sX[kK * PC];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, r16 = lane & 15, g4 = lane >> 4;
    const int wr = wave / 2 * (T / 2), wc = wave % 2 * (T / 2), lr = tid / Q, lc = (tid % Q) * 4;
    const int N = p.N, M = p.M, tm = (M + T - 1) / T, tn = (N + T - 1) / T;
    const int nb = (M + kCkptBlock - 1) / kCkptBlock;
    for (int tau = blockIdx.x; tau < tiles; tau += gridDim.x) {
        int rest = tau;
        const int m0 = rest % tm * T;
        rest /= tm;
        const int n0 = rest % tn * T;
        rest /= tn;
        const int pairs = p.dw[1] != nullptr ? 2 : 1, q = rest % pairs, j = rest / pairs;
        const float* dy = static_cast<const float*>(p.dy[q]);
        const int r0 = clampi(p.offsets[j], 0, p.cap), r1 = clampi(p.offsets[j + 1], r0, p.cap);
        float4 ry[F], rx[F];
        auto load = [&](int first) {
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const int r = first + i * (kThreads / Q) + lr;
                int a = r < r1 ? r : -1, b = a;
                if (p.src_of != nullptr && a >= 0) {
                    const int t = gathered(p.src_of, p.per, p.src_rows, r);
                    if (t < 0) a = b = -1;                   // adds nothing, whatever the other row holds
                    else (p.gather_dy ? a : b) = t;
                }
                ry[i] = a >= 0 && n0 + lc < N ? *reinterpret_cast<const float4*>(dy + (size_t)a * N + n0 + lc) : zero4();
                rx[i] = zero4();
                if (b >= 0 && m0 + lc < M) {
                    const size_t at = (size_t)b * M + m0 + lc;
                    if (p.x_scales != nullptr) {
                        const uint32_t c = *reinterpret_cast<const uint32_t*>(static_cast<const int8_t*>(p.x) + at);
                        const float s = p.x_scales[(size_t)b * nb + (m0 + lc) / kCkptBlock];
                        rx[i] = make_float4(code_value<0>(c) * s, code_value<1>(c) * s, code_value<2>(c) * s,
                                            code_value<3>(c) * s);
                    } else {
                        rx[i] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + at);
                    }
                }
            }
        };
        floatx4 acc[F][F] = {};
        load(r0);
        for (int r = r0; r < r1; r += kK) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < F; ++i) {
                *reinterpret_cast<float4*>(sY + (i * (kThreads / Q) + lr) * PC + lc) = ry[i];
                *reinterpret_cast<float4*>(sX + (i * (kThreads / Q) + lr) * PC + lc) = rx[i];
            }
            __syncthreads();
            if (r + kK < r1) load(r + kK);
#pragma unroll
            for (int k = 0; k < kK; k += 4) {
                float a[F], b[F];
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    a[i] = sY[(k + g4) * PC + wr + i * 16 + r16];
                    b[i] = sX[(k + g4) * PC + wc + i * 16 + r16];
                }
#pragma unroll
                for (int i = 0; i < F; ++i)
#pragma unroll
                    for (int jj = 0; jj < F; ++jj) acc[i][jj] = mma(a[i], b[jj], acc[i][jj]);
            }
        }
        const float* base = static_cast<const float*>(p.base[q]);
        float* dw = static_cast<float*>(p.dw[q]);
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int jj = 0; jj < F; ++jj)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = n0 + wr + i * 16 + g4 * 4 + e, m = m0 + wc + jj * 16 + r16;
                    if (n >= N || m >= M) continue;
                    const size_t at = ((size_t)j * N + n) * M + m;
                    dw[at] = base != nullptr ? acc[i][jj][e] + base[at] : acc[i][jj][e];
                }
    }
}

}  // namespace

hipError_t launch_ffn_ckpt_f32(const FfnArgs& a, hipStream_t stream) {
    static int per_cu = 0;
    return launch_persistent(gate_up_ckpt_kernel, kThreads, a, stream, &per_cu);
}
hipError_t launch_dgrad_f32(const FfnArgs& a, hipStream_t stream) {
    static int per_cu[2] = {0, 0};
    const long long large = (long long)a.E_loc * ((a.rows_hint + 63) / 64) * ((a.N + 63) / 64);
    if (large >= device_cu_count()) return launch_persistent(dgrad_kernel<64>, kThreads, a, stream, &per_cu[0]);
    return launch_persistent(dgrad_kernel<32>, kThreads, a, stream, &per_cu[1]);
}
template <int T>
hipError_t launch_wgrad_tiles(const WgradArgs& a, hipStream_t stream) {
    // (api.hip bounds dw)
    const int tiles = a.E_loc * (a.dw[1] != nullptr ? 2 : 1) * ((a.N + T - 1) / T) * ((a.M + T - 1) / T);
    const int most = device_cu_count() * 8;
    hipLaunchKernelGGL(wgrad_kernel<T>, dim3(tiles < most ? tiles : most), dim3(kThreads), 0, stream, a, tiles);
    return hipGetLastError();
}
hipError_t launch_wgrad_f32(const WgradArgs& a, hipStream_t stream) {
    const long long large = (long long)a.E_loc * (a.dw[1] != nullptr ? 2 : 1) * ((a.N + 63) / 64) * ((a.M + 63) / 64);
    return large >= device_cu_count() ? launch_wgrad_tiles<64>(a, stream) : launch_wgrad_tiles<32>(a, stream);
}

}  // namespace moeep
