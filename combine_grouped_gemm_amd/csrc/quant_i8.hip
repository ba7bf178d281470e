// Per-row int8 quantisation: of the tokens on their way to the experts
// (dispatch) and of expert-ordered rows (h between gate/up and down; weight
// rows, i.e. output channels).
//
// For a row v: amax = max |v|, scale = RN(amax / 127) in fp32 (at least the
// smallest normal number; 1 for amax = 0), code = v / scale rounded to the
// nearest integer, ties to even.  The quotient is rounded exactly: n =
// rint(v * (1 / scale)) is off by at most one step, and only next to a tie,
// and the remainder v - n * scale is exact in one fma (v and scale share the
// 24-bit grid of the larger one's last place, and |remainder| <= 0.51 scale),
// so comparing it with scale / 2 settles the code.  A row with a NaN or an
// infinity gets scale NaN and codes 0: every product with it is NaN.
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

// Code of v for the row scale s, rs = 1 / s (see the file comment); 0 when s is NaN.
__device__ __forceinline__ int code_of(float v, float s, float rs) {
    float n = rintf(v * rs);
    const float r = fmaf(-n, s, v), h = 0.5f * s;
    if (fabsf(r) >= h) {
        const bool odd = ((int)n & 1) != 0;
        if (r > h || (r == h && odd)) n += 1.0f;
        else if (r < -h || (r == -h && odd)) n -= 1.0f;
    }
    return s == s ? (int)n : 0;
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
    return (uint32_t)(a & 0xff) | ((uint32_t)(b & 0xff) << 8) | ((uint32_t)(c & 0xff) << 16) | ((uint32_t)d << 24);
}

// Eight consecutive values of a row: one 16-byte vector of bf16, two of fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void* row, int c, float (&f)[8]) {
    if constexpr (F32) {
        const uint4 a = static_cast<const uint4*>(row)[2 * c], b = static_cast<const uint4*>(row)[2 * c + 1];
        f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z);
        f[3] = __uint_as_float(a.w); f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
        f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    } else {
        const uint4 v = static_cast<const uint4*>(row)[c];
        f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
        f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
    }
}

__device__ __forceinline__ uint32_t amax8(const float (&f)[8], uint32_t m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(f[i]) & 0x7fffffffu;
        m = u > m ? u : m;
    }
    return m;
}

__device__ __forceinline__ uint2 codes8(const float (&f)[8], float s, float rs) {
    return make_uint2(pack4(code_of(f[0], s, rs), code_of(f[1], s, rs), code_of(f[2], s, rs), code_of(f[3], s, rs)),
                      pack4(code_of(f[4], s, rs), code_of(f[5], s, rs), code_of(f[6], s, rs), code_of(f[7], s, rs)));
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, d, kWave);
        v = o > v ? o : v;
    }
    return v;
}

// ---- dispatch: one block per token; the token is read once for its scale and
// once more (from cache) for its codes, which go to every local row.
constexpr int kTokThreads = 256;

template <bool F32>
__global__ __launch_bounds__(kTokThreads) void dispatch_i8_kernel(
    SegTable seg, int H, const int32_t* __restrict__ row_of, int K, int cap, uint8_t* __restrict__ xd,
    float* __restrict__ xd_scales) {
    __shared__ uint32_t s_max[kTokThreads / kWave];
    const int t = blockIdx.x, tid = threadIdx.x;
    const int32_t* rows = row_of + (size_t)t * K;
    bool any = false;
    for (int k = 0; k < K; ++k) any = any || (rows[k] >= 0 && rows[k] < cap);
    if (!any) return;
    int i = 0;
    for (int s = 1; s < seg.n; ++s) i += t >= seg.start[s] ? 1 : 0;
    const char* row = static_cast<const char*>(seg.ptr[i]) + (size_t)(t - seg.start[i]) * H * (F32 ? 4 : 2);
    uint32_t m = 0;
    for (int c = tid; c < H / 8; c += kTokThreads) {
        float f[8];
        load8<F32>(row, c, f);
        m = amax8(f, m);
    }
    m = wave_max_u32(m);
    if (tid % kWave == 0) s_max[tid / kWave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTokThreads / kWave; ++w) m = s_max[w] > m ? s_max[w] : m;
    const float s = row_scale(m), rs = 1.0f / s;
    for (int c = tid; c < H / 8; c += kTokThreads) {
        float f[8];
        load8<F32>(row, c, f);
        const uint2 q = codes8(f, s, rs);
        for (int k = 0; k < K; ++k) {
            const int r = rows[k];
            if (r >= 0 && r < cap) reinterpret_cast<uint2*>(xd + (size_t)r * H)[c] = q;
        }
    }
    for (int k = tid; k < K; k += kTokThreads) {
        const int r = rows[k];
        if (r >= 0 && r < cap) xd_scales[r] = s;
    }
}

// ---- expert-ordered rows: one wave per row over a persistent grid.  Valid
// rows are [offsets[0], offsets[E_loc]) of the contiguous layout, the first
// m[j] of each block of cap_e rows in the masked one, or all rows.
constexpr int kRowWaves = 4;

template <bool F32>
__global__ __launch_bounds__(kRowWaves * kWave) void quant_rows_kernel(QuantArgs p) {
    const int lane = threadIdx.x % kWave;
    const int wave = blockIdx.x * kRowWaves + threadIdx.x / kWave;
    int r0 = 0, r1 = p.cap;
    if (p.offsets != nullptr) {
        r0 = min(max(p.offsets[0], 0), p.cap);
        r1 = min(max(p.offsets[p.E_loc], r0), p.cap);
    }
    for (long long r = (long long)r0 + wave; r < r1; r += (long long)gridDim.x * kRowWaves) {
        if (p.m_counts != nullptr) {
            const int j = (int)(r / p.cap_e);
            if ((int)(r % p.cap_e) >= p.m_counts[j]) continue;
        }
        const char* row = static_cast<const char*>(p.x) + (size_t)r * p.cols * (F32 ? 4 : 2);
        uint32_t m = 0;
        for (int c = lane; c < p.cols / 8; c += kWave) {
            float f[8];
            load8<F32>(row, c, f);
            m = amax8(f, m);
        }
        const float s = row_scale(wave_max_u32(m)), rs = 1.0f / s;
        for (int c = lane; c < p.cols / 8; c += kWave) {
            float f[8];
            load8<F32>(row, c, f);
            reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.q) + (size_t)r * p.cols)[c] = codes8(f, s, rs);
        }
        if (lane == 0) p.scales[r] = s;
    }
}

}  // namespace

hipError_t launch_dispatch_i8(const SegTable& seg, int B, int H, bool f32, const int32_t* row_of, int K, void* xd,
                              float* xd_scales, int cap, hipStream_t stream) {
    if (B == 0) return hipSuccess;
    if (f32)
        hipLaunchKernelGGL(dispatch_i8_kernel<true>, dim3(B), dim3(kTokThreads), 0, stream, seg, H, row_of, K, cap,
                           static_cast<uint8_t*>(xd), xd_scales);
    else
        hipLaunchKernelGGL(dispatch_i8_kernel<false>, dim3(B), dim3(kTokThreads), 0, stream, seg, H, row_of, K, cap,
                           static_cast<uint8_t*>(xd), xd_scales);
    return hipGetLastError();
}

hipError_t launch_quant_rows(const QuantArgs& a, bool f32, hipStream_t stream) {
    if (a.cap == 0) return hipSuccess;
    const int want = (a.cap + kRowWaves - 1) / kRowWaves, most = device_cu_count() * 8;
    const dim3 grid(want < most ? want : most), block(kRowWaves * kWave);
    if (f32) hipLaunchKernelGGL(quant_rows_kernel<true>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(quant_rows_kernel<false>, grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace moeep
