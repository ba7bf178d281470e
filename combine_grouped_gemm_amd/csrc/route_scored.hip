// Scored routing: top-K experts by a score plus a balance bias, chosen inside
// the best expert groups, with gates taken from the scores.
//
// Per token, with logits l and bias b over E experts in G groups of E/G
// consecutive ids:
//   s_e = 1 / (1 + e^-l_e)  or  e^(l_e - max l) / sum e^(l - max l)
//   c_e = s_e + b_e                      (only the choice sees the bias)
//   a group's score is the sum of its group_top largest c; the topk_groups
//   best groups stay; the K largest c among their experts are the picks
//   gate_k = s_k (/ sum of the picked s) * scale
// An expert whose logit or bias is at or below the lowest finite bf16 value
// (-inf included) is out: it is never picked and a masked logit adds nothing
// to the softmax; slots left over get id -1 and gate 0.  Ties go to the lower
// id (group or expert); a NaN score ranks behind every number.
//
// Scores are compared in 64 bits: with a bias the order of two experts is not
// the order of their logits, and an 8192-token batch holds thousands of
// neighbours closer than fp32 sigmoids can tell apart.
//
// One wave per token, keys in LDS.
#include "device_common.hpp"
#include "launch.hpp"

namespace moeep {
namespace {

constexpr float kLowestBf16 = -3.3895313892515355e38f;    // -(2 - 2^-7) 2^127

// Order-preserving 64-bit key of a score: 0 for an expert that is out, 1 for
// NaN, then the numbers in ascending order (-0 ties with +0).
__device__ __forceinline__ uint64_t score_key(double c, bool on) {
    if (!on) return 0ull;
    if (c != c) return 1ull;
    const uint64_t u = (uint64_t)__double_as_longlong(c == 0.0 ? 0.0 : c);
    return (u >> 63) != 0 ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ double key_score(uint64_t k) {
    if (k == 1ull) return __longlong_as_double(0x7ff8000000000000ll);
    return __longlong_as_double((long long)((k >> 63) != 0 ? (k & 0x7fffffffffffffffull) : ~k));
}

__device__ __forceinline__ uint64_t shfl_xor_u64(uint64_t v, int m) {
    return (uint64_t)__shfl_xor((unsigned long long)v, m, kWave);
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
    return v;
}

// Largest key of s[0..n) and the lowest index that holds it, the same in
// every lane.
__device__ __forceinline__ uint64_t wave_argmax(const uint64_t* s, int n, int lane, int* at) {
    uint64_t best = 0;
    int idx = n;
    for (int i = lane; i < n; i += kWave)
        if (s[i] > best) { best = s[i]; idx = i; }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const uint64_t k = shfl_xor_u64(best, d);
        const int i = __shfl_xor(idx, d, kWave);
        if (k > best || (k == best && i < idx)) { best = k; idx = i; }
    }
    *at = idx;
    return best;
}

__device__ __forceinline__ float load_logit(const void* p, bool bf16, size_t i) {
    return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16)
                : static_cast<const float*>(p)[i];
}

__global__ __launch_bounds__(kWave) void route_scored_kernel(RouteScoredArgs p) {
    extern __shared__ uint64_t smem[];
    uint64_t* s_key = smem;                                       // E
    double* s_score = reinterpret_cast<double*>(smem + p.E);      // E
    uint64_t* s_group = smem + 2 * (size_t)p.E;                   // G
    double* s_val = reinterpret_cast<double*>(s_group + p.G);     // K
    int* s_id = reinterpret_cast<int*>(s_val + p.K);              // K
    const int t = blockIdx.x, lane = threadIdx.x;
    const size_t base = (size_t)t * p.E;

    float top = -INFINITY;
    if (!p.sigmoid) {
        for (int e = lane; e < p.E; e += kWave) {
            const float l = load_logit(p.logits, p.bf16, base + e);
            if (!(l <= kLowestBf16)) top = fmaxf(top, l);
        }
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
    }
    double sum = 0.0;
    for (int e = lane; e < p.E; e += kWave) {
        const float l = load_logit(p.logits, p.bf16, base + e);
        const bool on = !(l <= kLowestBf16);
        double s = 0.0;
        if (on) s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top);
        s_score[e] = s;
        sum += s;
    }
    sum = p.sigmoid ? 1.0 : wave_sum_f64(sum);
    for (int e = lane; e < p.E; e += kWave) {
        const float l = load_logit(p.logits, p.bf16, base + e);
        const float b = p.bias != nullptr ? p.bias[e] : 0.0f;
        const bool on = !(l <= kLowestBf16) && !(b <= kLowestBf16);
        const double s = p.sigmoid ? s_score[e] : s_score[e] / sum;
        s_score[e] = !(l <= kLowestBf16) ? s : 0.0;
        s_key[e] = score_key(s + (double)b, on);
    }
    __syncthreads();

    if (p.topk_groups < p.G) {
        const int S = p.E / p.G;
        for (int g = lane; g < p.G; g += kWave) {
            uint64_t k1 = 0, k2 = 0;                              // two best of the group
            for (int i = 0; i < S; ++i) {
                const uint64_t k = s_key[g * S + i];
                if (k > k1) { k2 = k1; k1 = k; }
                else if (k > k2) k2 = k;
            }
            uint64_t key = 0;
            if (k1 != 0)
                key = p.group_top == 1 || k2 == 0 ? k1 : score_key(key_score(k1) + key_score(k2), true);
            s_group[g] = key;
        }
        __syncthreads();
        // the groups that stay are taken out of s_group; the others keep their key
        for (int i = 0; i < p.topk_groups; ++i) {
            int g;
            const uint64_t k = wave_argmax(s_group, p.G, lane, &g);
            __syncthreads();
            if (k == 0) break;
            if (lane == 0) s_group[g] = 0;
            __syncthreads();
        }
        for (int e = lane; e < p.E; e += kWave)
            if (s_group[e / S] != 0) s_key[e] = 0;
        __syncthreads();
    }

    double total = 0.0;
    for (int k = 0; k < p.K; ++k) {
        int e;
        const uint64_t key = wave_argmax(s_key, p.E, lane, &e);
        const double s = key != 0 ? s_score[e] : 0.0;
        __syncthreads();
        if (lane == 0) {
            if (key != 0) s_key[e] = 0;
            s_val[k] = s;
            s_id[k] = key != 0 ? e : -1;
        }
        total += s;
        __syncthreads();
    }
    const int ld = p.K + p.n_shared;
    for (int k = lane; k < ld; k += kWave) {
        int id = p.E + (k - p.K);
        float w = 1.0f;
        if (k < p.K) {
            id = s_id[k];
            if (id >= 0 && p.map != nullptr) id = p.map[id];
            double v = s_val[k];
            // a NaN total is not zero: it reaches the gates
            if (p.renorm) v = total == 0.0 ? 0.0 : v / total;
            w = s_id[k] >= 0 ? (float)(v * (double)p.scale) : 0.0f;
        }
        p.ids[(size_t)t * ld + k] = id;
        p.w[(size_t)t * ld + k] = w;
    }
}

}  // namespace

hipError_t launch_route_scored(const RouteScoredArgs& a, hipStream_t stream) {
    if (a.B == 0) return hipSuccess;
    const size_t lds = (size_t)a.E * 16 + (size_t)a.G * 8 + (size_t)a.K * 12;
    hipLaunchKernelGGL(route_scored_kernel, dim3(a.B), dim3(kWave), lds, stream, a);
    return hipGetLastError();
}

}  // namespace moeep
