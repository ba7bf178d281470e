// Gradient of the routing weights back to the logits, for moe_route and
// moe_route_scored.
//
// With picks P of a token, dw the gradient of its weights w and s the scores:
//   softmax over the picks     dl_e = w_e (dw_e - sum_P w dw)               e in P
//   scored, renormalised       with the shares q = s / sum_P s: a_e = scale q_e (dw_e - sum_P q dw)
//     sigmoid                  dl_e = a_e (1 - s_e)                         e in P
//     softmax over all         dl_e = a_e (sum_P a = 0: the other experts have none)
//   scored, as they are        a_e = scale dw_e
//     sigmoid                  dl_e = a_e s_e (1 - s_e)                     e in P
//     softmax over all         dl_e = s_e ([e in P] a_e - sum_P s a)        every e that is not masked
// The forward call forms the shares in 64 bits, so weights and gradients of picks at -90 are
// ordinary numbers: where the scores' sum is too small for 32 bits they are taken relative to
// the largest pick's.  (Relative ones throughout cost 8192 tokens of 256 experts 0.7 us.)  Where
// the sum is zero in 64 bits too the weights are zeros and pass nothing.
// The choice itself is a step and passes no gradient, so neither does the bias.
//
// A wave takes a token.  Lane k holds pick k (picks beyond 64 in further
// registers' turns of a loop) and works on its own logit; the row of dlogits is
// then written once, each lane finding its experts among the picks (K compares an
// expert, by lane reads), so that no store depends on another.  1 - s of the
// sigmoid comes from e^-|l|, which does not cancel.
//
// In a graph, 8192 tokens of 256 experts, 8 picks: sigmoid 7.9 us, softmax over all 10.1 (not
// renormalised 11.3), of which 8.4 MB of dlogits take 1.3 at the rate of a fill and a launch 2 to 3;
// 64 tokens of 16, 2.8 us.  By the profiler 8.6 and 3.2.
#include "device_common.hpp"
#include "launch.hpp"
#include "moeep.h"

namespace moeep {
namespace {

constexpr int kWaves = 4;
constexpr int kMaxE = 1024;
// logits at or below the lowest finite bf16 value take their expert out
constexpr float kLow = -3.38953138925153547590470800371487866880e38f;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, kWave);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, kWave));
    return v;
}

template <bool BF16>
__device__ __forceinline__ float logit(const void* l, size_t i) {
    if constexpr (BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(l)[i] << 16);
    else return static_cast<const float*>(l)[i];
}

// 1 / (1 + e^-l) is zero in 64 bits from here down: e^-l passes the largest double, e^709.78271289
constexpr float kNoSigmoid = -0x1.62e43p9f;

// Renormalised scores whose sum lies below are formed anew: from here up a pick of 2^-26 of the
// sum and more is a normal number.
constexpr float kSmallSum = 0x1p-100f;

// s and 1 - s of the sigmoid
__device__ __forceinline__ void sigmoid2(float l, float& s, float& rest) {
    const float e = expf(-fabsf(l)), big = 1.0f / (1.0f + e), small = e * big;
    s = l >= 0.0f ? big : small;
    rest = l >= 0.0f ? small : big;
}

// RENORM: of a scored router; NP: picks a lane (K <= 64 NP)
template <bool BF16, int SCORE, bool RENORM, int NP>
__global__ __launch_bounds__(kWaves * kWave) void route_backward_kernel(RouteBwdArgs p) {
    __shared__ int s_inv[kMaxE];              // expert of a physical id, -1: none
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int E = p.E, K = p.K;
    if (p.map != nullptr) {
        for (int e = threadIdx.x; e < E; e += kWaves * kWave) s_inv[e] = -1;
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += kWaves * kWave) {
            const int q = p.map[e];
            if (q >= 0 && q < E) s_inv[q] = e;
        }
        __syncthreads();
    }
    for (long long t = (long long)blockIdx.x * kWaves + wave; t < p.B; t += (long long)gridDim.x * kWaves) {
        const size_t row = (size_t)t * E;
        // softmax over all: the row's maximum and sum
        float top = -INFINITY, total = 0.0f;
        if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
            for (int e = lane; e < E; e += kWave) {
                const float l = logit<BF16>(p.logits, row + e);
                if (!(l <= kLow)) top = fmaxf(top, l);
            }
            top = wave_max(top);
            for (int e = lane; e < E; e += kWave) {
                const float l = logit<BF16>(p.logits, row + e);
                if (!(l <= kLow)) total += expf(l - top);        // a NaN makes it NaN
            }
            total = wave_sum(total);
        }
        // the picks
        int at[NP];
        float s[NP], rest[NP], dw[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int k = i * kWave + lane;
            int e = -1;
            float l = 0.0f;
            dw[i] = 0.0f;
            if (k < K) {
                e = p.ids[(size_t)t * p.Kt + k];
                e = e >= 0 && e < E ? e : -1;
                if (p.map != nullptr && e >= 0) e = s_inv[e];
                if (e >= 0) {
                    l = logit<BF16>(p.logits, row + e);
                    if (SCORE != MOE_SCORE_PICKS && l <= kLow) e = -1;
                }
                if (e >= 0) dw[i] = p.dw[(size_t)t * p.Kt + k];
            }
            at[i] = e;
            s[i] = l;                          // the score follows
            rest[i] = 0.0f;
        }
        if constexpr (SCORE == MOE_SCORE_PICKS) {
            float m = -INFINITY, z = 0.0f;
#pragma unroll
            for (int i = 0; i < NP; ++i) m = fmaxf(m, at[i] >= 0 ? s[i] : -INFINITY);
            m = wave_max(m);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                s[i] = at[i] >= 0 ? expf(s[i] - m) : 0.0f;
                z += s[i];
            }
            z = wave_sum(z);
#pragma unroll
            for (int i = 0; i < NP; ++i) s[i] = at[i] >= 0 ? s[i] / z : 0.0f;
        } else {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                if constexpr (SCORE == MOE_SCORE_SIGMOID) sigmoid2(s[i], s[i], rest[i]);
                else s[i] = expf(s[i] - top) / total;
                if (at[i] < 0) s[i] = 0.0f;
            }
        }
        // a: the gradient of the logits (scores as they are, softmax over all: of the scores)
        float a[NP], sum = 0.0f;
        if constexpr (SCORE == MOE_SCORE_PICKS) {
#pragma unroll
            for (int i = 0; i < NP; ++i) sum += s[i] * dw[i];
            sum = wave_sum(sum);
#pragma unroll
            for (int i = 0; i < NP; ++i) a[i] = s[i] * (dw[i] - sum);
        } else if constexpr (RENORM) {
            float S = 0.0f;
#pragma unroll
            for (int i = 0; i < NP; ++i) S += s[i];
            S = wave_sum(S);
            bool none = false;
            if (S < kSmallSum) {               // the scores anew, over that of the largest pick
                float low = -INFINITY;
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    s[i] = at[i] >= 0 ? logit<BF16>(p.logits, row + at[i]) : -INFINITY;
                    low = fmaxf(low, s[i]);
                }
                low = wave_max(low);
                none = SCORE == MOE_SCORE_SIGMOID ? low <= kNoSigmoid
                                                  : exp((double)low - (double)top) / (double)total == 0.0;
                S = 0.0f;
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    // (so small a sigmoid is e^l)
                    s[i] = at[i] >= 0 ? expf(s[i] - low) : 0.0f;
                    S += s[i];
                }
                S = wave_sum(S);
            }
            // a NaN sum is not zero: it reaches the gradients, as it does the weights
            const bool some = S != 0.0f && !none;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                s[i] = some ? s[i] / S : 0.0f;
                sum += s[i] * dw[i];
            }
            sum = wave_sum(sum);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                a[i] = some ? p.scale * (s[i] * (dw[i] - sum)) : 0.0f;
                if constexpr (SCORE == MOE_SCORE_SIGMOID) a[i] *= rest[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                a[i] = p.scale * dw[i];
                if constexpr (SCORE == MOE_SCORE_SIGMOID) a[i] *= s[i] * rest[i];
            }
        }
        float all = 0.0f;                      // softmax over all, scores as they are: sum_P s a
        if constexpr (SCORE == MOE_SCORE_SOFTMAX && !RENORM) {
#pragma unroll
            for (int i = 0; i < NP; ++i) all += at[i] >= 0 ? s[i] * a[i] : 0.0f;
            all = wave_sum(all);
        }
        // whether experts that are no picks have a gradient
        const bool every = SCORE == MOE_SCORE_SOFTMAX &&
                           (!RENORM || __builtin_amdgcn_readfirstlane(total != total ? 1 : 0) != 0);
        for (int e = lane; e - lane < E; e += kWave) {
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int n = min(kWave, K - i * kWave);
                for (int k = 0; k < n; ++k) {
                    const int q = __builtin_amdgcn_readlane(at[i], k);
                    const float x = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(a[i]), k));
                    v += q == e ? x : 0.0f;
                }
            }
            if (e < E) {
                if (every) {
                    const float l = logit<BF16>(p.logits, row + e);
                    v = !(l <= kLow) ? expf(l - top) / total * (v - all) : 0.0f;
                }
                p.dlogits[row + e] = v;
            }
        }
    }
}

template <bool BF16, int SCORE, bool RENORM>
hipError_t launch_as(const RouteBwdArgs& a, hipStream_t stream) {
    const int need = (int)(((long long)a.B + kWaves - 1) / kWaves), most = device_cu_count() * 8;
    const dim3 grid(need < most ? need : most), block(kWaves * kWave);
    if (a.K <= 64) hipLaunchKernelGGL((route_backward_kernel<BF16, SCORE, RENORM, 1>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((route_backward_kernel<BF16, SCORE, RENORM, 16>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <int SCORE>
hipError_t launch_scored(const RouteBwdArgs& a, hipStream_t stream) {
    if (a.renorm) return a.bf16 ? launch_as<true, SCORE, true>(a, stream) : launch_as<false, SCORE, true>(a, stream);
    return a.bf16 ? launch_as<true, SCORE, false>(a, stream) : launch_as<false, SCORE, false>(a, stream);
}

}  // namespace

hipError_t launch_route_backward(const RouteBwdArgs& a, hipStream_t stream) {
    if (a.B == 0) return hipSuccess;
    if (a.score == MOE_SCORE_PICKS) return launch_as<false, MOE_SCORE_PICKS, false>(a, stream);      // (fp32 logits: api.hip)
    if (a.score == MOE_SCORE_SIGMOID) return launch_scored<MOE_SCORE_SIGMOID>(a, stream);
    return launch_scored<MOE_SCORE_SOFTMAX>(a, stream);
}

}  // namespace moeep
