// Internal launchers behind the C ABI.  Arguments have been validated by the
// caller (api.hip); each launcher only enqueues kernels on `stream` and
// returns the hipError_t of the launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moeep {

// Tokens of one launch of a kernel with up to 512 threads a token: a grid of 2^32
// threads or more is cut short without an error, so longer batches take several.
constexpr int kMostTokens = 1 << 22;

// part(first token, tokens) for each of the launches that B tokens take.
template <typename Part>
hipError_t launch_in_parts(int B, Part part) {
    for (long long b0 = 0; b0 < B; b0 += kMostTokens) {
        const hipError_t e = part((size_t)b0, B - b0 < kMostTokens ? (int)(B - b0) : kMostTokens);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// route.hip (map: optional (E) device table logical -> physical expert id; n_shared
// always-on slots appended to each output row, ids E.., gate 1)
hipError_t launch_route(const float* logits, int B, int E, int K, int32_t* ids, float* w,
                        const int32_t* map, int n_shared, hipStream_t stream);

// route_scored.hip
struct RouteScoredArgs {
    const void* logits;       // (B, E) fp32 or bf16
    const float* bias;        // (E) or nullptr
    const int32_t* map;       // (E) logical -> physical id, or nullptr
    int32_t* ids;             // (B, K + n_shared)
    float* w;
    float scale;
    int B, E, K, G, topk_groups, group_top, n_shared;
    bool bf16, sigmoid, renorm;
};
hipError_t launch_route_scored(const RouteScoredArgs& a, hipStream_t stream);

// placement.hip (host): balanced equal-size expert groups, see the file header
bool place_experts(const int64_t* load, int E, int G, int32_t* phys_of_logical);

// layout.hip
size_t layout_workspace_bytes(int B, int K, int E);
// moe_layout_noalloc: the layout workspace held by the library, one
// kLayoutScratchBytes array per GPU; layout_scratch_ptr gives the current
// GPU's copy (its device address, looked up once per GPU and cached)
constexpr size_t kLayoutScratchBytes = (size_t)4 << 20;
constexpr int kMaxDevices = 64;
hipError_t layout_scratch_ptr(void** out);
hipError_t launch_layout(const int32_t* ids, int B, int K, int E, int e_begin, int e_end,
                         int32_t* counts, int32_t* offsets, int32_t* row_of, int32_t* src_of,
                         int cap, void* ws, hipStream_t stream);
// fixed-capacity variant: local expert j owns rows [j*cap_e, (j+1)*cap_e); m (E_loc) gets
// min(count, cap_e)
hipError_t launch_layout_masked(const int32_t* ids, int B, int K, int E, int e_begin, int e_end,
                                int32_t* counts, int32_t* m, int32_t* row_of, int32_t* src_of,
                                int cap_e, void* ws, hipStream_t stream);

// dispatch.hip
constexpr int kMaxSeg = 64;
struct SegTable {
    const void* ptr[kMaxSeg];
    int start[kMaxSeg + 1];   // prefix sums of segment rows
    int n;

    // the same segments with tokens counted from b0 (earlier ones start below 0)
    SegTable from(size_t b0) const {
        SegTable t = *this;
        for (int s = 0; s <= n; ++s) t.start[s] -= (int)b0;
        return t;
    }
};
// kind: 0 = f32 copy, 1 = bf16 copy, 2 = bf16 -> fp8 quantise
hipError_t launch_dispatch(const SegTable& seg, int B, int H, int kind, const int32_t* row_of,
                           int K, void* xd, float* xd_scales, int cap, hipStream_t stream);

// quant_i8.hip: the same scatter with per-token int8 quantisation (x fp32 or bf16)
hipError_t launch_dispatch_i8(const SegTable& seg, int B, int H, bool f32, const int32_t* row_of, int K, void* xd,
                              float* xd_scales, int cap, hipStream_t stream);
struct QuantArgs {
    const void* x;            // (cap, cols) fp32 or bf16
    const int32_t* offsets;   // contiguous layout: (E_loc + 1), or nullptr
    const int32_t* m_counts;  // masked layout: (E_loc), or nullptr (both null: all rows)
    int E_loc, cap, cap_e, cols;
    void* q;                  // (cap, cols) int8
    float* scales;            // (cap)
};
hipError_t launch_quant_rows(const QuantArgs& a, bool f32, hipStream_t stream);

// combine.hip
// kind: 0 = f32 -> f32, 1 = bf16 -> bf16, 2 = bf16 -> f32
hipError_t launch_combine(const void* y, int kind, const int32_t* row_of, const float* w,
                          int B, int K, int H, void* out, int cap, hipStream_t stream);

// Division of a slot (below 2^31) by the slots of a token: q = umulhi(slot, mul) >> shift
// with l = ceil(log2 d), mul = floor(2^(31 + l) / d) + 1 and shift = l - 1: the multiplier
// is above 2^(31 + l) / d by at most 1, which moves the quotient by less than slot / 2^(31
// + l) < 1 / d, too little to reach the next integer.  d = 1: shift -1, the slot itself.
struct Divisor {
    uint32_t mul;
    int shift;
};
inline Divisor divisor_of(int d) {
    if (d <= 1) return Divisor{0, -1};
    int l = 1;
    while ((1 << l) < d) ++l;
    return Divisor{(uint32_t)((1ull << (31 + l)) / (unsigned)d + 1), l - 1};
}

// ffn kernels: shared argument block
struct FfnArgs {
    const void* a;            // activations (cap, Kdim)
    const float* a_scales;    // fp8: (cap, ceil(Kdim/128)); int8: (cap)
    const int32_t* offsets;   // contiguous layout: (E_loc + 1); nullptr for the masked layout
    const int32_t* m_counts;  // masked layout: (E_loc) valid rows of expert j, in [j*cap_e, ...)
    int cap_e;                // masked layout: rows per expert block (cap = E_loc * cap_e)
    int E_loc, cap, Kdim, N;  // N = output columns (I for gate/up, H for down)
    int ldw;                  // weight row pitch in elements (Kdim, or the packed pitch)
    const void* w0;           // gate or down (E_loc, N, ldw): rows of Kdim at pitch ldw
    const void* w1;           // up (gate/up only)
    const float* w0_scales;   // fp8: (E_loc, N, ceil(Kdim/128)); int8: (E_loc, N)
    const float* w1_scales;
    void* out;                // (cap, N)
    float* out_scales;        // fp8 h only: (cap, ceil(N/128))
    int rows_hint;            // cap / E_loc, picks the tile shape
    bool w_scales_pow2;       // fp8: every weight scale is a power of two
    bool out_f32;             // int8 down: fp32 outputs instead of bf16
    // gate/up of a training step: 8-bit checkpoints of g and u beside h
    int8_t* gate_q;           // (cap, N)
    int8_t* up_q;
    float* gate_s;            // (cap, ceil(N/128))
    float* up_s;
    // input gradients: out = a w0 + a2 w1 over the weights' rows (Kdim of them, N
    // columns at pitch ldw); with src_of row r of a is a's row src_of[r] / per
    const void* a2;
    const int32_t* src_of;    // (cap), or nullptr: row r itself
    int per, src_rows;
    Divisor per_div;          // by per
};

hipError_t launch_ffn_f32(const FfnArgs& a, bool gated, hipStream_t stream);   // ffn_f32.hip
hipError_t launch_ffn_bf16(const FfnArgs& a, bool gated, hipStream_t stream);  // ffn_bf16.hip
hipError_t launch_ffn_fp8(const FfnArgs& a, bool gated, hipStream_t stream);   // ffn_fp8.hip
hipError_t launch_ffn_i8(const FfnArgs& a, bool gated, hipStream_t stream);    // ffn_i8.hip

// the same with 8-bit checkpoints of g and u (gate_q ... up_s)
hipError_t launch_ffn_ckpt_f32(const FfnArgs& a, hipStream_t stream);          // grad_f32.hip
hipError_t launch_ffn_ckpt_bf16(const FfnArgs& a, hipStream_t stream);         // ffn_bf16.hip

// input gradients (a2, w1 may be null: one product)
hipError_t launch_dgrad_f32(const FfnArgs& a, hipStream_t stream);             // grad_f32.hip
hipError_t launch_dgrad_bf16(const FfnArgs& a, hipStream_t stream);            // dgrad_bf16.hip

// weight gradients: dw_j = base_j + sum over expert j's rows r of dy[r]^T x[r], for one
// or two dy that share x
struct WgradArgs {
    const void* dy[2];        // (rows, N); null where there are no rows, or no pair
    const void* x;            // (rows, M)
    const float* x_scales;    // checkpoint x: (rows, ceil(M/128)); else nullptr
    const int32_t* src_of;    // (cap): the gathered operand's row of r is src_of[r] / per
    int per, src_rows;        // src_rows: rows of the gathered operand
    Divisor per_div;          // by per
    bool gather_x, gather_dy;
    const int32_t* offsets;   // (E_loc + 1)
    int E_loc, cap, N, M;
    const void* base[2];      // (E_loc, N, M) or null; may be dw itself
    void* dw[2];              // dw[1] null: no pair
    bool dw_f32;
};
hipError_t launch_wgrad_f32(const WgradArgs& a, hipStream_t stream);           // grad_f32.hip
hipError_t launch_wgrad_bf16(const WgradArgs& a, hipStream_t stream);          // wgrad_bf16.hip

// ckpt.hip
struct CkptArgs {
    void* x;                  // (cap, cols) fp32 or bf16: read by the packing, written by the reading
    const int32_t* offsets;   // (E_loc + 1), or nullptr: all rows
    int E_loc, cap, cols;
    int8_t* q;                // (cap, cols)
    float* scales;            // (cap, ceil(cols/128))
};
hipError_t launch_checkpoint_rows(const CkptArgs& a, bool f32, hipStream_t stream);
hipError_t launch_checkpoint_values(const CkptArgs& a, bool f32, hipStream_t stream);

struct SwigluBwdArgs {
    const void* dh;           // (cap, I)
    const int8_t* gate_q;     // (cap, I)
    const int8_t* up_q;
    const float* gate_s;      // (cap, ceil(I/128))
    const float* up_s;
    const int32_t* row_of;    // (slots)
    const float* topk_w;      // (slots)
    void* dgate;              // (cap, I)
    void* dup;
    void* hw;
    float* dtopk_w;           // (slots)
    int cap, I;
    long long slots;
};
hipError_t launch_swiglu_backward(const SwigluBwdArgs& a, bool f32, hipStream_t stream);

// route_bwd.hip
struct RouteBwdArgs {
    const void* logits;       // (B, E) fp32 or bf16
    const int32_t* ids;       // (B, Kt)
    const float* dw;          // (B, Kt)
    const int32_t* map;       // (E) logical -> physical id, or nullptr
    float* dlogits;           // (B, E)
    float scale;
    int B, E, K, Kt, score;   // score: moe_score_t
    bool bf16, renorm;
};
hipError_t launch_route_backward(const RouteBwdArgs& a, hipStream_t stream);

int device_cu_count();   // api.hip: compute units of the current device (cached)

// pack.hip: rows of row_bytes bytes (a multiple of 4) copied to a pitch of
// ld_bytes (a multiple of 128, >= row_bytes), the padding zeroed
hipError_t launch_pack_rows(const void* src, long long n_rows, int row_bytes, int ld_bytes, void* dst,
                            hipStream_t stream);

}  // namespace moeep
