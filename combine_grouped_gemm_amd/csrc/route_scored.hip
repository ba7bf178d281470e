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
// neighbours closer than fp32 sigmoids can tell apart.  Few tokens need all of
// that, though, so the common kernel narrows in fp32 and settles in fp64:
//
//   A token is 16 lanes (a DPP row), four tokens a wave, and a group 16 / G of
//   them; a lane holds its share (rounded up) of the group's experts as 32-bit
//   keys (the score's leading bits, then the place in the lane), sorted once in
//   registers.  Groups are ranked by
//   DPP; K + 4 rounds of "row maximum, its owner shifts its list" give the
//   candidates, one to a lane.  Every candidate's score is then computed in 64
//   bits, one lane each, and ranked exactly, and its gate comes from that.
//   The answer stands if the K-th exact score lies above what any expert that
//   is no candidate can have (the last candidate's key plus the fp32 error),
//   and if the groups' cut is wider than that error; NaN and huge scores never
//   do.  Otherwise the wave does that token again in 64 bits from the start.
//
// Other shapes (E > 512, K > 12, a G that does not divide 16) go through that
// 64-bit routine, one wave a token, keys in LDS.
//
// Measured (MI355X, in a graph): one token of 256 experts, 8 groups, 5.3 us;
// 8192 of them 7.6-8.8 us (9.2 alone by the profiler; reading the logits would take
// 2 us).  Bound by the VALU: 1300 instructions a wave by the counter, two waves a
// SIMD, issuing 61% of the CUs' busy cycles, with little to hide the rest behind.
// 4093 tokens of 128 experts, softmax, bf16, 4.0-4.4 us (5.0 by the profiler).  More
// than 256 experts mean 32 keys a lane (149 VGPRs, scalars spilled, three waves a
// SIMD): 8192 tokens of 512 12.7-13.8 us (24.0 with logits read one by one), of 384,
// softmax, 13.1-15.0; 60 in 4 groups 5.5-6.4 (14 by the 64-bit routine).  The 64-bit
// routine costs four to five times as much: 256 experts with K = 12 7.5 us, K = 13
// 26.0, K = 22 37.1 (one token 5.2, 10.7, 15.6); 513 experts 42.5, 1024 95; 96 in 3
// groups 19.6; 512 with K = 22 71.9.
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

// The DPP move that CTRL names: partners lane ^ 1 (0xB1) and lane ^ 2 (0x4E),
// the mirrors of half a 16-lane row (0x141) and of a row (0x140), which join
// what those two have made uniform, and rotation of a row by r (0x120 + r).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
template <int CTRL>
__device__ __forceinline__ uint64_t dpp(uint64_t v) {
    return ((uint64_t)dpp<CTRL>((uint32_t)(v >> 32)) << 32) | dpp<CTRL>((uint32_t)v);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    return __longlong_as_double((long long)dpp<CTRL>((uint64_t)__double_as_longlong(v)));
}
// Reduction over a 16-lane row, the result in each of its lanes.
template <typename T, typename Op>
__device__ __forceinline__ T row_reduce(T v, Op op) {
    v = op(v, dpp<0xB1>(v));
    v = op(v, dpp<0x4E>(v));
    v = op(v, dpp<0x141>(v));
    return op(v, dpp<0x140>(v));
}
template <typename T>
__device__ __forceinline__ T row_max(T v) { return row_reduce(v, [](T a, T b) { return a > b ? a : b; }); }
template <typename T>
__device__ __forceinline__ T row_sum(T v) { return row_reduce(v, [](T a, T b) { return a + b; }); }

__device__ __forceinline__ uint64_t readlane_u64(uint64_t v, int l) {
    return ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), l) << 32) |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, l);
}

// LDS written by one lane of the wave, read by another.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Largest key of s[0..n) and the lowest index that holds it, the same in
// every lane.
__device__ __forceinline__ uint64_t wave_argmax(const uint64_t* s, int n, int lane, int* at) {
    uint64_t best = 0;
    int idx = n;
    for (int i = lane; i < n; i += kWave)
        if (s[i] > best) { best = s[i]; idx = i; }
    const uint64_t m = row_max(best);
    const uint64_t a = readlane_u64(m, 0), b = readlane_u64(m, 16), c = readlane_u64(m, 32), d = readlane_u64(m, 48);
    const uint64_t ab = a > b ? a : b, cd = c > d ? c : d, top = ab > cd ? ab : cd;
    const uint32_t none = 0xffffffffu;
    const uint32_t i = row_reduce(best == top && top != 0 ? (uint32_t)idx : none, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
    const uint32_t i0 = (uint32_t)__builtin_amdgcn_readlane((int)i, 0), i1 = (uint32_t)__builtin_amdgcn_readlane((int)i, 16);
    const uint32_t i2 = (uint32_t)__builtin_amdgcn_readlane((int)i, 32), i3 = (uint32_t)__builtin_amdgcn_readlane((int)i, 48);
    const uint32_t i01 = i0 < i1 ? i0 : i1, i23 = i2 < i3 ? i2 : i3;
    *at = (int)(i01 < i23 ? i01 : i23);
    return top;
}

__device__ __forceinline__ float load_logit(const void* p, bool bf16, size_t i) {
    return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16)
                : static_cast<const float*>(p)[i];
}

// Bytes of LDS that exact_token needs.
__host__ __device__ inline size_t exact_lds(int E, int G, int K) {
    return (size_t)E * 16 + (size_t)G * 8 + (size_t)((K + 1) / 2 * 2) * 12;
}

// One token by one wave, in 64 bits throughout.  smem: exact_lds bytes of the
// wave's own.
__device__ void exact_token(const RouteScoredArgs& p, int t, uint64_t* smem) {
    uint64_t* s_key = smem;                                       // E
    double* s_score = reinterpret_cast<double*>(smem + p.E);      // E
    uint64_t* s_group = smem + 2 * (size_t)p.E;                   // G
    double* s_val = reinterpret_cast<double*>(s_group + p.G);     // K
    int* s_id = reinterpret_cast<int*>(s_val + p.K);              // K
    const int lane = threadIdx.x % kWave;
    wave_lds_sync();                                              // an earlier token's reads are done
    const size_t base = (size_t)t * p.E;

    float top = -INFINITY;
    if (!p.sigmoid) {
        for (int e = lane; e < p.E; e += kWave) {
            const float l = load_logit(p.logits, p.bf16, base + e);
            if (!(l <= kLowestBf16)) top = fmaxf(top, l);
        }
        top = row_reduce(top, [](float x, float y) { return fmaxf(x, y); });
        top = fmaxf(fmaxf(__shfl(top, 0), __shfl(top, 16)), fmaxf(__shfl(top, 32), __shfl(top, 48)));
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
    if (!p.sigmoid) {
        sum = row_sum(sum);
        sum = (__shfl(sum, 0) + __shfl(sum, 16)) + (__shfl(sum, 32) + __shfl(sum, 48));
    }
    for (int e = lane; e < p.E; e += kWave) {
        const float l = load_logit(p.logits, p.bf16, base + e);
        const float b = p.bias != nullptr ? p.bias[e] : 0.0f;
        const bool on = !(l <= kLowestBf16) && !(b <= kLowestBf16);
        const double s = p.sigmoid ? s_score[e] : s_score[e] / sum;
        s_score[e] = !(l <= kLowestBf16) ? s : 0.0;
        s_key[e] = score_key(s + (double)b, on);
    }
    wave_lds_sync();

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
        wave_lds_sync();
        // the groups that stay are taken out of s_group; the others keep their key
        for (int i = 0; i < p.topk_groups; ++i) {
            int g;
            const uint64_t k = wave_argmax(s_group, p.G, lane, &g);
            wave_lds_sync();
            if (k == 0) break;
            if (lane == 0) s_group[g] = 0;
            wave_lds_sync();
        }
        for (int e = lane; e < p.E; e += kWave)
            if (s_group[e / S] != 0) s_key[e] = 0;
        wave_lds_sync();
    }

    double total = 0.0;
    for (int k = 0; k < p.K; ++k) {
        int e;
        const uint64_t key = wave_argmax(s_key, p.E, lane, &e);
        const double s = key != 0 ? s_score[e] : 0.0;
        wave_lds_sync();
        if (lane == 0) {
            if (key != 0) s_key[e] = 0;
            s_val[k] = s;
            s_id[k] = key != 0 ? e : -1;
        }
        total += s;
        wave_lds_sync();
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

__global__ __launch_bounds__(kWave) void route_scored_exact_kernel(RouteScoredArgs p) {
    extern __shared__ uint64_t smem[];
    exact_token(p, blockIdx.x, smem);
}

// ---- four tokens a wave (see the file comment)
constexpr int kRowWaves = 4;                // waves per block
constexpr int kExtra = 4;                   // candidates beyond K
constexpr int kMaxRowK = 16 - kExtra;

__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);                 // -0 becomes +0
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ (~(uint32_t)((int32_t)k >> 31) | 0x80000000u));
}

// e^x within 2^-22 of its value (down to where it underflows): the hardware's
// 2^x of the leading part of x / ln 2, times 1 + the rest.
__device__ __forceinline__ float exp_near(float x) {
    const float hi = 1.44269502f, lo = 1.925963e-8f;
    const float p = x * hi;
    const float r = fmaf(x, lo, fmaf(x, hi, -p));
    return __builtin_amdgcn_exp2f(p) * fmaf(r, 0.693147182f, 1.0f);
}

// How many groups have a larger score than this lane's (an equal one: a lower
// number); a group is `lanes` lanes that hold the same score.  The row is
// rotated in steps of a group.
template <typename T>
__device__ __forceinline__ int groups_ahead(T score, int lanes, int l16) {
    int n = 0;
    auto against = [&](T other, int r) {
        n += (int)((other > score) | ((other == score) & (((l16 - r) & 15) < l16)));
    };
#define MOEEP_AGAINST(r) against(dpp<0x120 + r>(score), r);
    if (lanes <= 8) { MOEEP_AGAINST(8) }
    if (lanes <= 4) { MOEEP_AGAINST(4) MOEEP_AGAINST(12) }
    if (lanes <= 2) { MOEEP_AGAINST(2) MOEEP_AGAINST(6) MOEEP_AGAINST(10) MOEEP_AGAINST(14) }
    if (lanes == 1) {
        MOEEP_AGAINST(1) MOEEP_AGAINST(3) MOEEP_AGAINST(5) MOEEP_AGAINST(7)
        MOEEP_AGAINST(9) MOEEP_AGAINST(11) MOEEP_AGAINST(13) MOEEP_AGAINST(15)
    }
#undef MOEEP_AGAINST
    return n;
}

// How a lane reads its share of the experts, EPL at most: one by one, in 16-byte
// pieces, or in pieces that fill all EPL registers.
enum Reads { kSingly, kPieces, kWhole };

template <int EPL, Reads READS, bool SIGMOID, bool BF16>
__global__ __launch_bounds__(kRowWaves * kWave) void route_scored_kernel(RouteScoredArgs p) {
    extern __shared__ uint64_t smem[];
    static_assert((EPL & (EPL - 1)) == 0 && EPL >= 4, "bitonic sort");
    constexpr uint32_t kPlace = EPL - 1;    // low key bits: the place in the lane, inverted
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int row = lane >> 4, l16 = lane & 15;
    const int t = (blockIdx.x * kRowWaves + wave) * 4 + row;
    const bool live = t < p.B;
    const size_t base = (size_t)(live ? t : p.B - 1) * p.E;       // idle rows repeat the last token
    const bool grouped = p.topk_groups < p.G;
    const int log_g = grouped ? __builtin_ctz(p.G) : 0;           // without groups the row is one
    const int lanes = 16 >> log_g, size = p.E >> log_g;           // of a group
    const int chunk = READS == kWhole ? EPL : (size + lanes - 1) / lanes;
    // the first expert of a lane; lanes behind a group's last expert have none
    auto first_expert = [&](int l) {
        return READS != kSingly ? l * chunk : (l >> (4 - log_g)) * size + (l & (lanes - 1)) * chunk;
    };
    const int e0 = first_expert(l16);
    const int mine = READS != kSingly ? chunk : min(chunk, size - (l16 & (lanes - 1)) * chunk);

    // ---- logits and biases of this lane's experts
    float lg[EPL], bs[EPL];
    if constexpr (READS != kSingly) {
        if constexpr (BF16) {
            const uint16_t* src = static_cast<const uint16_t*>(p.logits) + base + e0;
#pragma unroll
            for (int j = 0; j < EPL; j += 8) {
                uint4 v = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
                if (READS == kWhole || j < chunk) v = *reinterpret_cast<const uint4*>(src + j);
                lg[j] = bf16_lo(v.x); lg[j + 1] = bf16_hi(v.x); lg[j + 2] = bf16_lo(v.y); lg[j + 3] = bf16_hi(v.y);
                lg[j + 4] = bf16_lo(v.z); lg[j + 5] = bf16_hi(v.z); lg[j + 6] = bf16_lo(v.w); lg[j + 7] = bf16_hi(v.w);
            }
        } else {
            const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.logits) + base + e0);
#pragma unroll
            for (int j = 0; j < EPL; j += 4) {
                float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (READS == kWhole || j < chunk) v = src[j / 4];
                lg[j] = v.x; lg[j + 1] = v.y; lg[j + 2] = v.z; lg[j + 3] = v.w;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) lg[j] = j < mine ? load_logit(p.logits, BF16, base + e0 + j) : -INFINITY;
    }
    if (p.bias != nullptr) {
        if constexpr (READS != kSingly) {
            const float4* src = reinterpret_cast<const float4*>(p.bias + e0);
#pragma unroll
            for (int j = 0; j < EPL; j += 4) {
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (READS == kWhole || j < chunk) v = src[j / 4];
                bs[j] = v.x; bs[j + 1] = v.y; bs[j + 2] = v.z; bs[j + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j) bs[j] = j < mine ? p.bias[e0 + j] : 0.0f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) bs[j] = 0.0f;
    }

    // ---- softmax: the largest logit and the sum, in 64 bits (gates and exact scores need them)
    float top = -INFINITY;
    double sum = 1.0, inv = 1.0;
    double ex[SIGMOID ? 1 : EPL];
    if constexpr (!SIGMOID) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) top = fmaxf(top, lg[j] <= kLowestBf16 ? -INFINITY : lg[j]);
        top = row_reduce(top, [](float x, float y) { return fmaxf(x, y); });
        if (top == -INFINITY) top = 0.0f;                        // nothing but masked logits
        sum = 0.0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            ex[j] = exp((double)lg[j] - (double)top);            // 0 for a masked logit
            sum += ex[j];
        }
        sum = row_sum(sum);
        inv = 1.0 / sum;
    }

    // ---- keys.  Error of a 32-bit score against the exact one: for the sigmoid
    // exp_near's 2^-22 (weighed by 1 - s), the sum's 2^-24 and the reciprocal's
    // last place, 2^-23; softmax is rounded once; adding the bias rounds once more.
    // In all less than 2^-21 of s <= 1 and of c: `rel`, and `abs_err` where a
    // bias may cancel s (without one only what underflows is lost).  No branches
    // here: they would cost more than what they skip.
    const float rel = 0x1p-21f, abs_err = p.bias != nullptr ? 0x1p-21f : 1e-37f;
    uint32_t key[EPL];
    float c1 = -INFINITY, c2 = -INFINITY;   // the lane's two best
    bool odd = false;                       // a score that is no ordinary number
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const bool off = (lg[j] <= kLowestBf16) | (bs[j] <= kLowestBf16);
        float c;
        if constexpr (SIGMOID) c = __builtin_amdgcn_rcpf(1.0f + exp_near(-lg[j])) + bs[j];
        else c = (float)(ex[j] * inv + (double)bs[j]);
        odd |= !off & !(fabsf(c) < 1e30f);
        key[j] = off ? 0u : ((order_key(c) & ~kPlace) | (kPlace - j));
        c = off ? -INFINITY : c;
        c2 = __builtin_amdgcn_fmed3f(c1, c2, c);
        c1 = fmaxf(c1, c);
    }

    // ---- sorted in the lane, largest first
#pragma unroll
    for (int k = 2; k <= EPL; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1)
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int l = i ^ j;
                if (l > i) {
                    const uint32_t hi = key[i] > key[l] ? key[i] : key[l], lo = key[i] > key[l] ? key[l] : key[i];
                    const bool down = (i & k) == 0;
                    key[i] = down ? hi : lo;
                    key[l] = down ? lo : hi;
                }
            }

    // an expert's score s and choice c in 64 bits
    auto exact_score = [&](int e, double* s) {
        const double l = (double)load_logit(p.logits, BF16, base + e);
        const double b = p.bias != nullptr ? (double)p.bias[e] : 0.0;
        *s = SIGMOID ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top) / sum;
        return *s + b;
    };
    // what no expert's exact score exceeds whose key is k or less
    auto key_bound = [&](uint32_t k) {
        const float up = key_value(k | kPlace);                   // without the place's bits, rounded up
        return (double)up + (double)fabsf(up) * rel + abs_err;
    };

    // ---- groups
    bool ok = true;
    if (grouped) {
        auto join = [&](float o1, float o2) {
            c2 = fmaxf(fminf(c1, o1), fmaxf(c2, o2));
            c1 = fmaxf(c1, o1);
        };
        if (lanes > 1) join(dpp<0xB1>(c1), dpp<0xB1>(c2));
        if (lanes > 2) join(dpp<0x4E>(c1), dpp<0x4E>(c2));
        if (lanes > 4) join(dpp<0x141>(c1), dpp<0x141>(c2));
        const float second = (p.group_top == 2) & (c2 != -INFINITY) ? c2 : 0.0f;
        const float score = c1 + second;
        // of the two terms, which may cancel
        const float terms = c1 != -INFINITY ? fabsf(c1) + fabsf(second) : 0.0f;
        bool kept = groups_ahead(score, lanes, l16) < p.topk_groups;
        // the cut between the last group kept and the first one dropped
        const float least = -row_max(kept & (c1 != -INFINITY) ? -score : -INFINITY);
        const float most = row_max(kept ? -INFINITY : score);
        const float slack = 2.0f * (row_max(terms) * rel + 2.0f * abs_err);
        ok = (most == -INFINITY) | (least - most > slack);
        if (ballot64(!ok) != 0) {
            // too near to tell (a token in five thousand; one in an 8192-token batch
            // would hold up the kernel by half if it went through exact_token):
            // the same with exact scores, of each lane's three leading experts,
            // among which its two best are if the fourth is far enough behind
            double x1 = -(double)INFINITY, x2 = x1;
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                double s, c = -(double)INFINITY;
                if (key[q] != 0) c = exact_score(e0 + (int)(kPlace - (key[q] & kPlace)), &s);
                x2 = fmax(fmin(x1, c), x2);
                x1 = fmax(x1, c);
            }
            const bool sure = (key[3] == 0) | (x2 > key_bound(key[3]));
            auto join64 = [&](double o1, double o2) {
                x2 = fmax(fmin(x1, o1), fmax(x2, o2));
                x1 = fmax(x1, o1);
            };
            if (lanes > 1) join64(dpp<0xB1>(x1), dpp<0xB1>(x2));
            if (lanes > 2) join64(dpp<0x4E>(x1), dpp<0x4E>(x2));
            if (lanes > 4) join64(dpp<0x141>(x1), dpp<0x141>(x2));
            const double exact = x1 + ((p.group_top == 2) & (x2 != -(double)INFINITY) ? x2 : 0.0);
            const bool kept64 = groups_ahead(exact, lanes, l16) < p.topk_groups;
            kept = ok ? kept : kept64;
            ok |= ((ballot64(!sure) >> (row * 16)) & 0xffffu) == 0;
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = kept ? key[j] : 0u;
    }

    // ---- candidates: candidate i in lane i of the row
    const int n_cand = min(p.K + kExtra, 16);
    int ce = -1;                            // its expert
    uint32_t last = 0;
    for (int i = 0; i < n_cand; ++i) {
        last = row_max(key[0]);
        const uint32_t owners = (uint32_t)(ballot64(key[0] == last) >> (row * 16)) & 0xffffu;
        const int first = __builtin_ctz(owners | 0x10000u);
        // the owner's list moves up by one: a bit select by a mask whose origin the
        // compiler does not see (it made a register index of the plain choice,
        // fifty instructions a place)
        uint32_t up = l16 == first ? 0xffffffffu : 0u;
        asm("" : "+v"(up));
        if ((l16 == i) & (last != 0)) ce = first_expert(first) + (int)(kPlace - (last & kPlace));
#pragma unroll
        for (int j = 0; j + 1 < EPL; ++j) key[j] = (key[j + 1] & up) | (key[j] & ~up);
        key[EPL - 1] &= ~up;
    }

    // ---- their exact scores and ranks
    double s = 0.0, c = -INFINITY;
    if (ce >= 0) c = exact_score(ce, &s);
    const uint32_t id = (uint32_t)ce;       // -1 ranks last
    int rank = 0;
    auto behind = [&](double oc, uint32_t oid) { rank += (int)((oc > c) | ((oc == c) & (oid < id))); };
#define MOEEP_BEHIND(r) behind(dpp<0x120 + r>(c), dpp<0x120 + r>(id));
    MOEEP_BEHIND(1) MOEEP_BEHIND(2) MOEEP_BEHIND(3) MOEEP_BEHIND(4) MOEEP_BEHIND(5)
    MOEEP_BEHIND(6) MOEEP_BEHIND(7) MOEEP_BEHIND(8) MOEEP_BEHIND(9) MOEEP_BEHIND(10)
    MOEEP_BEHIND(11) MOEEP_BEHIND(12) MOEEP_BEHIND(13) MOEEP_BEHIND(14) MOEEP_BEHIND(15)
#undef MOEEP_BEHIND
    const bool pick = ce >= 0 && rank < p.K;
    if (last != 0) {                        // there may be experts that are no candidates
        const double kth = -row_max(pick ? -c : -(double)INFINITY);
        ok = ok && kth > key_bound(last);
    }
    // every lane votes, whatever its ok: a NaN among the candidates makes kth, and so
    // ok, differ between the lanes of a row
    const bool strange = ((ballot64(odd) >> (row * 16)) & 0xffffu) != 0;
    ok = ok & !strange;

    const double total = row_sum(pick ? s : 0.0);
    const int ld = p.K + p.n_shared;
    int32_t* ids = p.ids + (size_t)t * ld;
    float* w = p.w + (size_t)t * ld;
    if (live && ok) {
        if (pick) {
            const double v = p.renorm ? (total == 0.0 ? 0.0 : s / total) : s;
            ids[rank] = p.map != nullptr ? p.map[ce] : ce;
            w[rank] = (float)(v * (double)p.scale);
        }
        const int found = __popc((uint32_t)(ballot64(pick) >> (row * 16)) & 0xffffu);
        if (l16 >= found && l16 < p.K) {
            ids[l16] = -1;
            w[l16] = 0.0f;
        }
        for (int k = p.K + l16; k < ld; k += 16) {
            ids[k] = p.E + (k - p.K);
            w[k] = 1.0f;
        }
    }
    uint64_t again = ballot64(live && !ok && l16 == 0);
    uint64_t* ws = smem + wave * (exact_lds(p.E, p.G, p.K) / 8);
    while (again != 0) {
        const int first = __builtin_ctzll(again);
        again &= again - 1;
        exact_token(p, __builtin_amdgcn_readlane(t, first), ws);
    }
}

template <int EPL, Reads READS>
hipError_t launch_rows(const RouteScoredArgs& a, hipStream_t stream) {
    const int per_block = kRowWaves * 4;
    const dim3 grid((a.B + per_block - 1) / per_block), block(kRowWaves * kWave);
    const size_t lds = kRowWaves * exact_lds(a.E, a.G, a.K);
    if (a.sigmoid && a.bf16) hipLaunchKernelGGL((route_scored_kernel<EPL, READS, true, true>), grid, block, lds, stream, a);
    else if (a.sigmoid) hipLaunchKernelGGL((route_scored_kernel<EPL, READS, true, false>), grid, block, lds, stream, a);
    else if (a.bf16) hipLaunchKernelGGL((route_scored_kernel<EPL, READS, false, true>), grid, block, lds, stream, a);
    else hipLaunchKernelGGL((route_scored_kernel<EPL, READS, false, false>), grid, block, lds, stream, a);
    return hipGetLastError();
}

hipError_t launch_tokens(const RouteScoredArgs& a, hipStream_t stream) {
    // a group is a whole number of a row's 16 lanes, or there are none
    const bool grouped = a.topk_groups < a.G;
    if (a.E <= 512 && a.K <= kMaxRowK && (!grouped || 16 % a.G == 0)) {
        const int lanes = grouped ? 16 / a.G : 16, size = grouped ? a.E / a.G : a.E;
        const int per_lane = (size + lanes - 1) / lanes;
        // E a multiple of 16: every lane has the same number of experts
        const bool pieces = a.E % 16 == 0 && per_lane % (a.bf16 ? 8 : 4) == 0 &&
                            ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.bias)) & 15u) == 0;
        if (per_lane == 8 && pieces) return launch_rows<8, kWhole>(a, stream);
        if (per_lane == 16 && pieces) return launch_rows<16, kWhole>(a, stream);
        if (per_lane <= 8) return launch_rows<8, kSingly>(a, stream);
        if (per_lane <= 16) return launch_rows<16, kSingly>(a, stream);
        return pieces ? launch_rows<32, kPieces>(a, stream) : launch_rows<32, kSingly>(a, stream);
    }
    hipLaunchKernelGGL(route_scored_exact_kernel, dim3(a.B), dim3(kWave), exact_lds(a.E, a.G, a.K), stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route_scored(const RouteScoredArgs& a, hipStream_t stream) {
    const int ld = a.K + a.n_shared;
    return launch_in_parts(a.B, [&](size_t b0, int n) {
        RouteScoredArgs part = a;
        part.B = n;
        part.logits = static_cast<const char*>(a.logits) + b0 * a.E * (a.bf16 ? 2 : 4);
        part.ids = a.ids + b0 * ld;
        part.w = a.w + b0 * ld;
        return launch_tokens(part, stream);
    });
}

}  // namespace moeep
