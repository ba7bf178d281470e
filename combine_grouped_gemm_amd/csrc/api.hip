// C ABI of libmoeep: host-side argument checks, then kernel launches on the
// caller's stream.  Nothing here allocates, synchronises or copies from the
// device; a failed check returns before anything is enqueued.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "launch.hpp"
#include "moeep.h"

static_assert(MOE_LAYOUT_NOALLOC_SCRATCH_BYTES == moeep::kLayoutScratchBytes,
              "the header states the library's layout scratch size");

namespace moeep {

int device_cu_count() {
    static thread_local int cached_dev = -1, cached_cus = 0;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 256;
    if (dev != cached_dev) {
        int cus = 0;
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 1)
            cus = 256;
        cached_dev = dev;
        cached_cus = cus;
    }
    return cached_cus;
}

}  // namespace moeep

namespace {

thread_local char g_last_error[512] = "";

moe_status_t fail(moe_status_t s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return s;
}

moe_status_t launched(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "%s: kernel launch failed: %s", what, hipGetErrorString(e));
    g_last_error[0] = '\0';
    return MOE_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define REQUIRE(cond, ...)                                        \
    do {                                                          \
        if (!(cond)) return fail(MOE_ERR_INVALID_ARG, __VA_ARGS__); \
    } while (0)

moe_status_t check_route_shape(int B, int E, int K) {
    REQUIRE(B >= 0, "B must be >= 0 (got %d)", B);
    REQUIRE(E >= 1 && E <= 1024, "E must be in [1, 1024] (got %d)", E);
    REQUIRE(K >= 1 && K <= E, "K must be in [1, E] (got K=%d, E=%d)", K, E);
    REQUIRE((long long)B * K <= 0x7fffffffLL && (long long)B * E <= 0x7fffffffLL,
            "B*K and B*E must fit in int32");
    return MOE_OK;
}

// Where the rows of each local expert are: the contiguous layout's offsets
// (E_local + 1), or the masked layout's valid-row counts m (E_local) with
// fixed blocks of cap_e rows.
struct Rows {
    const int32_t* offsets;
    const int32_t* m;
    int cap_e;
};

// names: whether the two sizes are H and I (else those of a weight, out and in)
moe_status_t check_ffn_common(const void* a, Rows rows, int E_local, int cap_rows,
                              int H, int I, moe_dtype_t act_dt, moe_dtype_t w_dt, bool names = true) {
    // a buffer of no rows has no address to give
    REQUIRE((a || cap_rows == 0) && (rows.offsets || rows.m), "null activation or row-count pointer");
    REQUIRE(E_local >= 1 && E_local <= 1024, "E_local must be in [1, 1024] (got %d)", E_local);
    REQUIRE(cap_rows >= 0, "cap_rows must be >= 0");
    // rows move in 16-byte pieces: 8 elements (bf16, fp32), 16 for fp8 and int8
    const int q = act_dt == MOE_FP8_E4M3 || act_dt == MOE_INT8 ? 16 : 8;
    REQUIRE(H >= q && H % q == 0 && I >= q && I % q == 0,
            names ? "H and I must be positive multiples of %d for this dtype (got H=%d, I=%d)"
                  : "out_dim and in_dim must be positive multiples of %d (got %d, %d)",
            q, H, I);
    REQUIRE((long long)cap_rows * (H > I ? H : I) <= 0x7fffffffLL * 4LL, "cap_rows * H too large");
    REQUIRE(aligned16(a), "activation pointer must be 16-byte aligned");
    const bool ok = (act_dt == MOE_F32 && w_dt == MOE_F32) || (act_dt == MOE_BF16 && w_dt == MOE_BF16) ||
                    (act_dt == MOE_FP8_E4M3 && (w_dt == MOE_FP8_E4M3 || w_dt == MOE_FP8_E4M3_PO2)) ||
                    (act_dt == MOE_INT8 && w_dt == MOE_INT8);
    if (!ok) return fail(MOE_ERR_UNSUPPORTED, "unsupported (act_dt, w_dt) = (%d, %d)", act_dt, w_dt);
    // 2^14 per product of two codes: the int32 sums are exact up to this length
    if (act_dt == MOE_INT8)
        REQUIRE(H <= MOE_INT8_MAX_COLS && I <= MOE_INT8_MAX_COLS, "int8 H and I must be at most %d (got H=%d, I=%d)",
                MOE_INT8_MAX_COLS, H, I);
    return MOE_OK;
}

moe_status_t check_y_dtype(moe_dtype_t act_dt, moe_dtype_t y_dt) {
    const bool ok = (act_dt == MOE_F32 && y_dt == MOE_F32) || (act_dt == MOE_BF16 && y_dt == MOE_BF16) ||
                    (act_dt == MOE_FP8_E4M3 && y_dt == MOE_BF16) ||
                    (act_dt == MOE_INT8 && (y_dt == MOE_BF16 || y_dt == MOE_F32));
    if (!ok) return fail(MOE_ERR_UNSUPPORTED, "unsupported (act_dt, y_dt) = (%d, %d)", act_dt, y_dt);
    return MOE_OK;
}

moeep::FfnArgs ffn_args(const void* a, const float* a_scales, Rows rows, int E_local,
                        int cap_rows, int Kdim, int N, const void* w0, const void* w1,
                        const float* w0s, const float* w1s, void* out, float* out_scales,
                        int expected_rows, moe_dtype_t w_dt, int ldw) {
    moeep::FfnArgs f;
    f.w_scales_pow2 = w_dt == MOE_FP8_E4M3_PO2;
    f.out_f32 = false;
    f.gate_q = f.up_q = nullptr;
    f.gate_s = f.up_s = nullptr;
    f.a2 = nullptr;
    f.src_of = nullptr;
    f.per = 1;
    f.per_div = moeep::divisor_of(1);
    f.src_rows = 0;
    f.ldw = ldw;
    f.a = a;
    f.a_scales = a_scales;
    f.offsets = rows.offsets;
    f.m_counts = rows.m;
    f.cap_e = rows.cap_e;
    f.E_loc = E_local;
    f.cap = cap_rows;
    f.Kdim = Kdim;
    f.N = N;
    f.w0 = w0;
    f.w1 = w1;
    f.w0_scales = w0s;
    f.w1_scales = w1s;
    f.out = out;
    f.out_scales = out_scales;
    f.rows_hint = expected_rows > 0 ? expected_rows : cap_rows / E_local;
    return f;
}

hipError_t run_ffn(const moeep::FfnArgs& f, moe_dtype_t act_dt, bool gated, hipStream_t stream) {
    if (f.cap == 0) return hipSuccess;
    switch (act_dt) {
        case MOE_F32: return moeep::launch_ffn_f32(f, gated, stream);
        case MOE_BF16: return moeep::launch_ffn_bf16(f, gated, stream);
        case MOE_INT8: return moeep::launch_ffn_i8(f, gated, stream);
        default: return moeep::launch_ffn_fp8(f, gated, stream);
    }
}

size_t elem_size(moe_dtype_t d) { return d == MOE_F32 ? 4 : d == MOE_BF16 ? 2 : 1; }

// Row pitch (elements) of packed weights: whole 128-byte lines, plus one line
// when the row length is a multiple of 4 KiB (rows exactly 4 KiB apart
// stream markedly slower than rows one line further apart).
int packed_ld(int cols, size_t esz) {
    size_t bytes = ((size_t)cols * esz + 127) / 128 * 128;
    if (bytes % 4096 == 0) bytes += 128;
    return (int)(bytes / esz);
}

// a weight dtype argument: the element type, and whether the rows sit at the packed pitch
struct WType {
    moe_dtype_t dt;
    bool packed;
};
WType split_w(moe_dtype_t w_dt) { return WType{w_dt & ~MOE_W_PACKED, (w_dt & MOE_W_PACKED) != 0}; }
int weight_ld(WType wt, int cols) { return wt.packed ? packed_ld(cols, elem_size(wt.dt)) : cols; }

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

size_t ffn_workspace_bytes(int cap_rows, int I, moe_dtype_t act_dt) {
    if (cap_rows < 0 || I < 1) return 0;
    // int8: h as gate/up writes it (bf16), its codes and its row scales
    if (act_dt == MOE_INT8)
        return round256((size_t)cap_rows * I * 2) + round256((size_t)cap_rows * I) +
               round256((size_t)cap_rows * sizeof(float));
    size_t bytes = round256((size_t)cap_rows * I * elem_size(act_dt));
    if (act_dt == MOE_FP8_E4M3) bytes += round256((size_t)cap_rows * (((size_t)I + 127) / 128) * sizeof(float));
    return bytes;
}

moe_status_t ffn_gate_up(const void* xd, const float* xd_scales, Rows rows,
                             int E_local, int cap_rows, int H, int I, moe_dtype_t act_dt,
                             const void* w_gate, const void* w_up, const float* w_gate_scales,
                             const float* w_up_scales, moe_dtype_t w_dt, void* h, float* h_scales,
                             int expected_rows, hipStream_t stream) {
    const WType wt = split_w(w_dt);
    moe_status_t s = check_ffn_common(xd, rows, E_local, cap_rows, H, I, act_dt, wt.dt);
    if (s != MOE_OK) return s;
    REQUIRE(w_gate && w_up && (h || cap_rows == 0), "null weight or h pointer");
    REQUIRE(aligned16(w_gate) && aligned16(w_up) && aligned16(h), "weights and h must be 16-byte aligned");
    if (act_dt == MOE_FP8_E4M3)
        REQUIRE(((xd_scales && h_scales) || cap_rows == 0) && w_gate_scales && w_up_scales,
                "fp8 needs all scale pointers");
    if (act_dt == MOE_INT8)
        REQUIRE((xd_scales || cap_rows == 0) && w_gate_scales && w_up_scales,
                "int8 needs the row and channel scale pointers");
    auto f = ffn_args(xd, xd_scales, rows, E_local, cap_rows, H, I, w_gate, w_up, w_gate_scales,
                      w_up_scales, h, h_scales, expected_rows, wt.dt, weight_ld(wt, H));
    return launched(run_ffn(f, act_dt, true, stream), "ffn gate/up");
}

moe_status_t ffn_down(const void* h, const float* h_scales, Rows rows, int E_local,
                          int cap_rows, int H, int I, moe_dtype_t act_dt, const void* w_down,
                          const float* w_down_scales, moe_dtype_t w_dt, void* y, moe_dtype_t y_dt,
                          int expected_rows, hipStream_t stream) {
    const WType wt = split_w(w_dt);
    moe_status_t s = check_ffn_common(h, rows, E_local, cap_rows, H, I, act_dt, wt.dt);
    if (s != MOE_OK) return s;
    s = check_y_dtype(act_dt, y_dt);
    if (s != MOE_OK) return s;
    REQUIRE(w_down && (y || cap_rows == 0), "null weight or y pointer");
    REQUIRE(aligned16(w_down) && aligned16(y), "weights and y must be 16-byte aligned");
    if (act_dt == MOE_FP8_E4M3)
        REQUIRE((h_scales || cap_rows == 0) && w_down_scales, "fp8 needs all scale pointers");
    if (act_dt == MOE_INT8)
        REQUIRE((h_scales || cap_rows == 0) && w_down_scales, "int8 needs the row and channel scale pointers");
    auto f = ffn_args(h, h_scales, rows, E_local, cap_rows, I, H, w_down, nullptr, w_down_scales,
                      nullptr, y, nullptr, expected_rows, wt.dt, weight_ld(wt, I));
    f.out_f32 = act_dt == MOE_INT8 && y_dt == MOE_F32;
    return launched(run_ffn(f, act_dt, false, stream), "ffn down");
}

// rows of (cap_rows, cols) named by `rows` (all when it names none)
moe_status_t quant_rows(const void* x, moe_dtype_t x_dt, Rows rows, int E_local, int cap_rows, int cols, int8_t* q,
                        float* scales, hipStream_t stream) {
    if (x_dt != MOE_F32 && x_dt != MOE_BF16) return fail(MOE_ERR_UNSUPPORTED, "unsupported x_dt %d", x_dt);
    REQUIRE(cap_rows >= 0, "cap_rows must be >= 0");
    REQUIRE(cols >= 16 && cols % 16 == 0 && cols <= MOE_INT8_MAX_COLS,
            "cols must be a positive multiple of 16, at most %d (got %d)", MOE_INT8_MAX_COLS, cols);
    if (rows.offsets || rows.m)
        REQUIRE(E_local >= 1 && E_local <= 1024, "E_local must be in [1, 1024] (got %d)", E_local);
    if (cap_rows > 0) {
        REQUIRE(x && q && scales, "null x, q or scales pointer");
        REQUIRE(aligned16(x) && aligned16(q), "x and q must be 16-byte aligned");
        const size_t n = (size_t)cap_rows * cols;
        const char* x0 = static_cast<const char*>(x);
        const char* q0 = reinterpret_cast<const char*>(q);
        REQUIRE(q0 + n <= x0 || x0 + n * elem_size(x_dt) <= q0, "x and q must not overlap");
    }
    moeep::QuantArgs a;
    a.x = x;
    a.offsets = rows.offsets;
    a.m_counts = rows.m;
    a.E_loc = E_local;
    a.cap = cap_rows;
    a.cap_e = rows.cap_e;
    a.cols = cols;
    a.q = q;
    a.scales = scales;
    return launched(moeep::launch_quant_rows(a, x_dt == MOE_F32, stream), "moe_quant_rows");
}

// ---- training step ---------------------------------------------------------------
moe_status_t check_train_dtype(moe_dtype_t act_dt, moe_dtype_t w_dt) {
    if ((act_dt != MOE_F32 && act_dt != MOE_BF16) || w_dt != act_dt)
        return fail(MOE_ERR_UNSUPPORTED, "unsupported (act_dt, w_dt) = (%d, %d): training takes F32 or BF16", act_dt, w_dt);
    return MOE_OK;
}

moe_status_t check_gather(bool gathers, int slots_per_token, int src_rows) {
    if (!gathers) return MOE_OK;
    REQUIRE(slots_per_token >= 1 && slots_per_token <= 1024, "slots_per_token must be in [1, 1024] (got %d)",
            slots_per_token);
    REQUIRE(src_rows >= 0, "src_rows must be >= 0 (got %d)", src_rows);
    return MOE_OK;
}

// whether two buffers share no byte (a null or an empty one shares none)
bool apart(const void* a, size_t na, const void* b, size_t nb) {
    const char *p = static_cast<const char*>(a), *q = static_cast<const char*>(b);
    return !p || !q || na == 0 || nb == 0 || p + na <= q || q + nb <= p;
}

struct Span {
    const void* p;
    size_t bytes;
};
bool apart(const Span& a, const Span& b) { return apart(a.p, a.bytes, b.p, b.bytes); }

// whether the outputs share no byte with each other or with an input: blocks of a launch
// write them while others still read
bool outputs_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        for (const Span* q = o + 1; q != outs.end(); ++q)
            if (!apart(*o, *q)) return false;
        for (const Span& i : ins)
            if (!apart(*o, i)) return false;
    }
    return true;
}

Span ints(const int32_t* p, long long n) { return Span{p, (size_t)n * sizeof(int32_t)}; }
// fp32 scales of rows of checkpoints
Span ckpt_scales(const float* p, int rows, int cols) {
    return Span{p, (size_t)rows * (((size_t)cols + MOE_CKPT_BLOCK - 1) / MOE_CKPT_BLOCK) * sizeof(float)};
}

// (columns are counted in ints, a tile's last ones past the end too)
constexpr int kTrainCols = 1 << 24;

// checkpoints of rows: x to q and scales, or back
moe_status_t checkpoint(void* x, moe_dtype_t x_dt, const int32_t* offsets, int E_local, int cap_rows, int cols,
                        int8_t* q, float* scales, bool write, hipStream_t stream) {
    if (x_dt != MOE_F32 && x_dt != MOE_BF16)
        return fail(MOE_ERR_UNSUPPORTED, "unsupported %s %d", write ? "x_dt" : "out_dt", x_dt);
    REQUIRE(cap_rows >= 0, "cap_rows must be >= 0");
    REQUIRE(cols >= 8 && cols % 8 == 0 && cols <= kTrainCols, "cols must be a positive multiple of 8, at most %d (got %d)",
            kTrainCols, cols);
    if (offsets) REQUIRE(E_local >= 1 && E_local <= 1024, "E_local must be in [1, 1024] (got %d)", E_local);
    if (cap_rows > 0) {
        REQUIRE(x && q && scales, "null %s, q or scales pointer", write ? "x" : "out");
        // (rows of codes are whole 8-byte pieces: a range of rows of a checkpoint is one too)
        REQUIRE(aligned16(x), "%s must be 16-byte aligned", write ? "x" : "out");
        REQUIRE((reinterpret_cast<uintptr_t>(q) & 7u) == 0, "q must be 8-byte aligned");
        const size_t n = (size_t)cap_rows * cols;
        const Span values{x, n * elem_size(x_dt)}, codes{q, n}, sc = ckpt_scales(scales, cap_rows, cols);
        const Span off = ints(offsets, (long long)E_local + 1);
        REQUIRE(write ? outputs_apart({codes, sc}, {values, off}) : outputs_apart({values}, {codes, sc, off}),
                write ? "q and scales must not overlap each other, x or offsets" : "out must not overlap q, scales or offsets");
    }
    moeep::CkptArgs a;
    a.x = x;
    a.offsets = offsets;
    a.E_loc = E_local;
    a.cap = cap_rows;
    a.cols = cols;
    a.q = q;
    a.scales = scales;
    const bool f32 = x_dt == MOE_F32;
    if (write) return launched(moeep::launch_checkpoint_rows(a, f32, stream), "moe_checkpoint_rows");
    return launched(moeep::launch_checkpoint_values(a, f32, stream), "moe_checkpoint_values");
}

moe_status_t grouped_ffn(const void* xd, const float* xd_scales, Rows rows,
                             int E_local, int cap_rows, int H, int I, moe_dtype_t act_dt,
                             const void* w_gate, const void* w_up, const void* w_down,
                             const float* w_gate_scales, const float* w_up_scales,
                             const float* w_down_scales, moe_dtype_t w_dt, void* y, moe_dtype_t y_dt,
                             void* ws, size_t ws_bytes, int expected_rows, hipStream_t stream) {
    moe_status_t s = check_ffn_common(xd, rows, E_local, cap_rows, H, I, act_dt, split_w(w_dt).dt);
    if (s != MOE_OK) return s;
    s = check_y_dtype(act_dt, y_dt);
    if (s != MOE_OK) return s;
    REQUIRE(ws, "null workspace");
    REQUIRE((reinterpret_cast<uintptr_t>(ws) & 255u) == 0, "workspace must be 256-byte aligned");
    const size_t need = ffn_workspace_bytes(cap_rows, I, act_dt);
    REQUIRE(ws_bytes >= need, "workspace too small: %zu < %zu bytes", ws_bytes, need);
    void* h = ws;
    float* h_scales = nullptr;
    if (act_dt == MOE_FP8_E4M3)
        h_scales = reinterpret_cast<float*>(static_cast<char*>(ws) + round256((size_t)cap_rows * I));
    if (act_dt == MOE_INT8) {
        // everything the three calls check is checked before the first is enqueued
        REQUIRE(w_gate && w_up && w_down && (y || cap_rows == 0), "null weight or y pointer");
        REQUIRE(aligned16(w_gate) && aligned16(w_up) && aligned16(w_down) && aligned16(y),
                "weights and y must be 16-byte aligned");
        REQUIRE((xd_scales || cap_rows == 0) && w_gate_scales && w_up_scales && w_down_scales,
                "int8 needs the row and channel scale pointers");
        int8_t* hq = reinterpret_cast<int8_t*>(static_cast<char*>(ws) + round256((size_t)cap_rows * I * 2));
        float* hs = reinterpret_cast<float*>(hq + round256((size_t)cap_rows * I));
        s = ffn_gate_up(xd, xd_scales, rows, E_local, cap_rows, H, I, act_dt, w_gate, w_up, w_gate_scales,
                        w_up_scales, w_dt, h, nullptr, expected_rows, stream);
        if (s != MOE_OK) return s;
        s = quant_rows(h, MOE_BF16, rows, E_local, cap_rows, I, hq, hs, stream);
        if (s != MOE_OK) return s;
        return ffn_down(hq, hs, rows, E_local, cap_rows, H, I, act_dt, w_down, w_down_scales, w_dt, y, y_dt,
                        expected_rows, stream);
    }
    s = ffn_gate_up(xd, xd_scales, rows, E_local, cap_rows, H, I, act_dt, w_gate, w_up,
                        w_gate_scales, w_up_scales, w_dt, h, h_scales, expected_rows, stream);
    if (s != MOE_OK) return s;
    return ffn_down(h, h_scales, rows, E_local, cap_rows, H, I, act_dt, w_down, w_down_scales,
                        w_dt, y, y_dt, expected_rows, stream);
}


}  // namespace

extern "C" {

const char* moe_status_string(moe_status_t s) {
    switch (s) {
        case MOE_OK: return "MOE_OK";
        case MOE_ERR_INVALID_ARG: return "MOE_ERR_INVALID_ARG";
        case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED";
        case MOE_ERR_HIP: return "MOE_ERR_HIP";
    }
    return "unknown status";
}

const char* moe_last_error(void) { return g_last_error; }

const char* moe_version(void) { return "libmoeep 0.1 (gfx950)"; }

moe_status_t moe_route(const float* logits, int B, int E, int K, int32_t* topk_ids, float* topk_w,
                       hipStream_t stream) {
    moe_status_t s = check_route_shape(B, E, K);
    if (s != MOE_OK) return s;
    if (B > 0) REQUIRE(logits && topk_ids && topk_w, "null pointer argument");
    return launched(moeep::launch_route(logits, B, E, K, topk_ids, topk_w, nullptr, 0, stream), "moe_route");
}

moe_status_t moe_route_mapped(const float* logits, int B, int E, int K, const int32_t* phys_of_logical,
                              int32_t* topk_ids, float* topk_w, hipStream_t stream) {
    moe_status_t s = check_route_shape(B, E, K);
    if (s != MOE_OK) return s;
    REQUIRE(phys_of_logical, "null phys_of_logical");
    if (B > 0) REQUIRE(logits && topk_ids && topk_w, "null pointer argument");
    return launched(moeep::launch_route(logits, B, E, K, topk_ids, topk_w, phys_of_logical, 0, stream),
                    "moe_route_mapped");
}

moe_status_t moe_route_shared(const float* logits, int B, int E, int K, int n_shared, int32_t* ids,
                              float* w, hipStream_t stream) {
    moe_status_t s = check_route_shape(B, E, K);
    if (s != MOE_OK) return s;
    REQUIRE(n_shared >= 0 && E + n_shared <= 1024, "need 0 <= n_shared and E + n_shared <= 1024");
    REQUIRE((long long)B * (K + n_shared) <= 0x7fffffffLL, "B*(K+n_shared) must fit in int32");
    if (B > 0) REQUIRE(logits && ids && w, "null pointer argument");
    return launched(moeep::launch_route(logits, B, E, K, ids, w, nullptr, n_shared, stream),
                    "moe_route_shared");
}

moe_status_t moe_route_scored(const void* logits, moe_dtype_t logits_dt, const float* bias, int B, int E, int K,
                              moe_score_t score, int n_groups, int topk_groups, int group_top, int renorm,
                              float scale, const int32_t* phys_of_logical, int n_shared, int32_t* ids, float* w,
                              hipStream_t stream) {
    moe_status_t s = check_route_shape(B, E, K);
    if (s != MOE_OK) return s;
    if (logits_dt != MOE_F32 && logits_dt != MOE_BF16)
        return fail(MOE_ERR_UNSUPPORTED, "unsupported logits_dt %d", logits_dt);
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)
        return fail(MOE_ERR_UNSUPPORTED, "unsupported score %d", score);
    REQUIRE(n_groups >= 1 && E % n_groups == 0, "n_groups must divide E (got E=%d, n_groups=%d)", E, n_groups);
    REQUIRE(topk_groups >= 1 && topk_groups <= n_groups, "topk_groups must be in [1, n_groups] (got %d of %d)",
            topk_groups, n_groups);
    REQUIRE(group_top == 1 || group_top == 2, "group_top must be 1 or 2 (got %d)", group_top);
    REQUIRE(K <= topk_groups * (E / n_groups), "K=%d exceeds the %d experts of %d groups", K,
            topk_groups * (E / n_groups), topk_groups);
    REQUIRE(std::isfinite(scale), "scale must be finite");
    REQUIRE(n_shared >= 0 && n_shared <= 1024 - E, "need 0 <= n_shared and E + n_shared <= 1024");
    REQUIRE((long long)B * (K + n_shared) <= 0x7fffffffLL, "B*(K+n_shared) must fit in int32");
    if (B > 0) REQUIRE(logits && ids && w, "null pointer argument");
    moeep::RouteScoredArgs a;
    a.logits = logits;
    a.bias = bias;
    a.map = phys_of_logical;
    a.ids = ids;
    a.w = w;
    a.scale = scale;
    a.B = B;
    a.E = E;
    a.K = K;
    a.G = n_groups;
    a.topk_groups = topk_groups;
    a.group_top = group_top;
    a.n_shared = n_shared;
    a.bf16 = logits_dt == MOE_BF16;
    a.sigmoid = score == MOE_SCORE_SIGMOID;
    a.renorm = renorm != 0;
    return launched(moeep::launch_route_scored(a, stream), "moe_route_scored");
}

moe_status_t moe_eplb_place(const int64_t* load, int E, int n_groups, int32_t* phys_of_logical) {
    REQUIRE(E >= 1 && E <= 1024, "E must be in [1, 1024] (got %d)", E);
    REQUIRE(n_groups >= 1 && E % n_groups == 0, "n_groups must divide E (got E=%d, n_groups=%d)", E,
            n_groups);
    REQUIRE(load && phys_of_logical, "null load or phys_of_logical");
    int64_t total = 0;     // group totals and their differences stay within it
    for (int e = 0; e < E; ++e) {
        REQUIRE(load[e] >= 0, "load[%d] < 0", e);
        REQUIRE(load[e] <= INT64_MAX - total, "the loads' total must fit in int64");
        total += load[e];
    }
    moeep::place_experts(load, E, n_groups, phys_of_logical);
    g_last_error[0] = '\0';
    return MOE_OK;
}

size_t moe_layout_workspace_bytes(int B, int K, int E) {
    // 0 for sizes moe_layout rejects (B * K past int32 included)
    if (B < 0 || K < 1 || E < 1 || (long long)B * K > 0x7fffffffLL) return 0;
    return moeep::layout_workspace_bytes(B, K, E);
}

moe_status_t moe_layout(const int32_t* topk_ids, int B, int K, int E, int e_begin, int e_end,
                        int32_t* counts, int32_t* offsets, int32_t* row_of, int32_t* src_of,
                        int cap_rows, void* ws, size_t ws_bytes, hipStream_t stream) {
    moe_status_t s = check_route_shape(B, E, K);
    if (s != MOE_OK) return s;
    REQUIRE(e_begin >= 0 && e_begin < e_end && e_end <= E,
            "need 0 <= e_begin < e_end <= E (got %d, %d, E=%d)", e_begin, e_end, E);
    REQUIRE(cap_rows >= 0, "cap_rows must be >= 0");
    REQUIRE(counts && offsets && ws, "null counts, offsets or workspace");
    if (B > 0) REQUIRE(topk_ids && row_of, "null topk_ids or row_of");
    if (cap_rows > 0) REQUIRE(src_of, "null src_of");
    REQUIRE((reinterpret_cast<uintptr_t>(ws) & 255u) == 0, "workspace must be 256-byte aligned");
    REQUIRE(ws_bytes >= moeep::layout_workspace_bytes(B, K, E),
            "workspace too small: %zu < %zu bytes", ws_bytes, moeep::layout_workspace_bytes(B, K, E));
    return launched(moeep::launch_layout(topk_ids, B, K, E, e_begin, e_end, counts, offsets, row_of,
                                         src_of, cap_rows, ws, stream),
                    "moe_layout");
}

moe_status_t moe_layout_noalloc(const int32_t* topk_ids, int B, int K, int E, int e_begin, int e_end,
                                int32_t* counts, int32_t* offsets, int32_t* row_of, int32_t* src_of,
                                int cap_rows, hipStream_t stream) {
    moe_status_t s = check_route_shape(B, E, K);
    if (s != MOE_OK) return s;
    REQUIRE(e_begin >= 0 && e_begin < e_end && e_end <= E,
            "need 0 <= e_begin < e_end <= E (got %d, %d, E=%d)", e_begin, e_end, E);
    REQUIRE(cap_rows >= 0, "cap_rows must be >= 0");
    REQUIRE(counts && offsets, "null counts or offsets");
    if (B > 0) REQUIRE(topk_ids && row_of, "null topk_ids or row_of");
    if (cap_rows > 0) REQUIRE(src_of, "null src_of");
    const size_t need = moeep::layout_workspace_bytes(B, K, E);
    REQUIRE(need <= moeep::kLayoutScratchBytes,
            "moe_layout_noalloc: B=%d, K=%d, E=%d needs %zu bytes of layout workspace, more than the "
            "library's %zu (use moe_layout with a caller workspace)",
            B, K, E, need, moeep::kLayoutScratchBytes);
    void* ws = nullptr;
    const hipError_t e = moeep::layout_scratch_ptr(&ws);
    if (e != hipSuccess)
        return fail(MOE_ERR_HIP, "moe_layout_noalloc: no device address for the layout scratch: %s",
                    hipGetErrorString(e));
    return launched(moeep::launch_layout(topk_ids, B, K, E, e_begin, e_end, counts, offsets, row_of,
                                         src_of, cap_rows, ws, stream),
                    "moe_layout_noalloc");
}

moe_status_t moe_layout_masked(const int32_t* topk_ids, int B, int K, int E, int e_begin, int e_end,
                               int32_t* counts, int32_t* m, int32_t* row_of, int32_t* src_of,
                               int cap_per_expert, void* ws, size_t ws_bytes, hipStream_t stream) {
    moe_status_t s = check_route_shape(B, E, K);
    if (s != MOE_OK) return s;
    REQUIRE(e_begin >= 0 && e_begin < e_end && e_end <= E,
            "need 0 <= e_begin < e_end <= E (got %d, %d, E=%d)", e_begin, e_end, E);
    REQUIRE(cap_per_expert >= 1, "cap_per_expert must be >= 1 (got %d)", cap_per_expert);
    REQUIRE((long long)(e_end - e_begin) * cap_per_expert <= 0x7fffffffLL,
            "E_local * cap_per_expert must fit in int32");
    REQUIRE(counts && m && src_of && ws, "null counts, m, src_of or workspace");
    if (B > 0) REQUIRE(topk_ids && row_of, "null topk_ids or row_of");
    REQUIRE((reinterpret_cast<uintptr_t>(ws) & 255u) == 0, "workspace must be 256-byte aligned");
    REQUIRE(ws_bytes >= moeep::layout_workspace_bytes(B, K, E),
            "workspace too small: %zu < %zu bytes", ws_bytes, moeep::layout_workspace_bytes(B, K, E));
    return launched(moeep::launch_layout_masked(topk_ids, B, K, E, e_begin, e_end, counts, m, row_of,
                                                src_of, cap_per_expert, ws, stream),
                    "moe_layout_masked");
}

moe_status_t moe_dispatch(const void* const* seg_x, const int32_t* seg_rows, int n_seg,
                          moe_dtype_t x_dt, int H, const int32_t* row_of, int K, void* xd,
                          moe_dtype_t xd_dt, float* xd_scales, int cap_rows, hipStream_t stream) {
    REQUIRE(n_seg >= 1 && n_seg <= MOE_MAX_SEGMENTS, "n_seg must be in [1, %d]", MOE_MAX_SEGMENTS);
    REQUIRE(seg_x && seg_rows, "null segment tables");
    REQUIRE(K >= 1 && K <= 1024, "K must be in [1, 1024]");
    // 16-byte pieces: 8 elements; fp8 and int8 rows feed GEMMs that need 16
    const int q = xd_dt == MOE_FP8_E4M3 || xd_dt == MOE_INT8 ? 16 : 8;
    REQUIRE(H >= q && H % q == 0, "H must be a positive multiple of %d for this dtype (got %d)", q, H);
    REQUIRE(cap_rows >= 0, "cap_rows must be >= 0");
    int kind;
    if (x_dt == MOE_F32 && xd_dt == MOE_F32) kind = 0;
    else if (x_dt == MOE_BF16 && xd_dt == MOE_BF16) kind = 1;
    else if (x_dt == MOE_BF16 && xd_dt == MOE_FP8_E4M3) kind = 2;
    else if ((x_dt == MOE_BF16 || x_dt == MOE_F32) && xd_dt == MOE_INT8) kind = 3;
    else return fail(MOE_ERR_UNSUPPORTED, "unsupported dispatch (x_dt, xd_dt) = (%d, %d)", x_dt, xd_dt);
    if (kind == 3)
        REQUIRE(H <= MOE_INT8_MAX_COLS, "int8 H must be at most %d (got %d)", MOE_INT8_MAX_COLS, H);
    moeep::SegTable seg;
    seg.n = n_seg;
    seg.start[0] = 0;
    long long B = 0;
    for (int i = 0; i < n_seg; ++i) {
        REQUIRE(seg_rows[i] >= 0, "seg_rows[%d] < 0", i);
        if (seg_rows[i] > 0) {
            REQUIRE(seg_x[i] != nullptr, "seg_x[%d] is null", i);
            REQUIRE(aligned16(seg_x[i]), "seg_x[%d] must be 16-byte aligned", i);
        }
        seg.ptr[i] = seg_x[i];
        B += seg_rows[i];
        REQUIRE(B * K <= 0x7fffffffLL, "total tokens * K must fit in int32");
        seg.start[i + 1] = (int)B;
    }
    if (B > 0) {
        REQUIRE(row_of && (xd || cap_rows == 0), "null row_of or xd");
        REQUIRE(aligned16(xd), "xd must be 16-byte aligned");
        if (kind == 2) REQUIRE(xd_scales || cap_rows == 0, "fp8 dispatch needs xd_scales");
        if (kind == 3) REQUIRE(xd_scales || cap_rows == 0, "int8 dispatch needs xd_scales");
    }
    if (kind == 3)
        return launched(moeep::launch_dispatch_i8(seg, (int)B, H, x_dt == MOE_F32, row_of, K, xd, xd_scales, cap_rows,
                                                  stream),
                        "moe_dispatch");
    return launched(moeep::launch_dispatch(seg, (int)B, H, kind, row_of, K, xd, xd_scales, cap_rows, stream),
                    "moe_dispatch");
}

size_t moe_ffn_workspace_bytes(int cap_rows, int I, moe_dtype_t act_dt) {
    return ffn_workspace_bytes(cap_rows, I, act_dt);
}

static bool packable_dtype(moe_dtype_t w_dt) {
    return w_dt == MOE_F32 || w_dt == MOE_BF16 || w_dt == MOE_FP8_E4M3 || w_dt == MOE_FP8_E4M3_PO2 ||
           w_dt == MOE_INT8;
}

int moe_weight_ld(int cols, moe_dtype_t w_dt) {
    if (cols < 1 || cols > (1 << 24) || !packable_dtype(w_dt & ~MOE_W_PACKED)) return -1;
    return packed_ld(cols, elem_size(w_dt & ~MOE_W_PACKED));
}

size_t moe_packed_weight_bytes(int E_local, int rows, int cols, moe_dtype_t w_dt) {
    const int ld = moe_weight_ld(cols, w_dt);
    if (ld < 0 || E_local < 0 || rows < 0) return 0;
    return (size_t)E_local * (size_t)rows * (size_t)ld * elem_size(w_dt & ~MOE_W_PACKED);
}

moe_status_t moe_pack_weights(const void* w, int E_local, int rows, int cols, moe_dtype_t w_dt,
                              void* w_packed, hipStream_t stream) {
    const moe_dtype_t dt = w_dt & ~MOE_W_PACKED;
    if (!packable_dtype(dt)) return fail(MOE_ERR_UNSUPPORTED, "unsupported weight dtype %d", w_dt);
    REQUIRE(E_local >= 0 && rows >= 0, "E_local and rows must be >= 0");
    REQUIRE(cols >= 8 && cols % 8 == 0 && cols <= (1 << 24), "cols must be a positive multiple of 8 (got %d)", cols);
    if ((long long)E_local * rows == 0) {
        g_last_error[0] = '\0';
        return MOE_OK;
    }
    REQUIRE(w && w_packed, "null weight pointer");
    REQUIRE(aligned16(w) && aligned16(w_packed), "weights must be 16-byte aligned");
    const size_t esz = elem_size(dt);
    const size_t row_bytes = (size_t)cols * esz, ld_bytes = (size_t)packed_ld(cols, esz) * esz;
    const long long n_rows = (long long)E_local * rows;
    const char* s0 = static_cast<const char*>(w);
    const char* d0 = static_cast<const char*>(w_packed);
    REQUIRE(d0 + (size_t)n_rows * ld_bytes <= s0 || s0 + (size_t)n_rows * row_bytes <= d0,
            "w and w_packed must not overlap");
    return launched(moeep::launch_pack_rows(w, n_rows, (int)row_bytes, (int)ld_bytes, w_packed, stream),
                    "moe_pack_weights");
}

moe_status_t moe_quant_rows(const void* x, moe_dtype_t x_dt, const int32_t* offsets, int E_local, int cap_rows,
                            int cols, int8_t* q, float* scales, hipStream_t stream) {
    return quant_rows(x, x_dt, Rows{offsets, nullptr, 0}, E_local, cap_rows, cols, q, scales, stream);
}

moe_status_t moe_ffn_gate_up(const void* xd, const float* xd_scales, const int32_t* offsets,
                             int E_local, int cap_rows, int H, int I, moe_dtype_t act_dt,
                             const void* w_gate, const void* w_up, const float* w_gate_scales,
                             const float* w_up_scales, moe_dtype_t w_dt, void* h, float* h_scales,
                             int expected_rows, hipStream_t stream) {
    return ffn_gate_up(xd, xd_scales, Rows{offsets, nullptr, 0}, E_local, cap_rows, H, I, act_dt,
                       w_gate, w_up, w_gate_scales, w_up_scales, w_dt, h, h_scales, expected_rows,
                       stream);
}

moe_status_t moe_ffn_down(const void* h, const float* h_scales, const int32_t* offsets, int E_local,
                          int cap_rows, int H, int I, moe_dtype_t act_dt, const void* w_down,
                          const float* w_down_scales, moe_dtype_t w_dt, void* y, moe_dtype_t y_dt,
                          int expected_rows, hipStream_t stream) {
    return ffn_down(h, h_scales, Rows{offsets, nullptr, 0}, E_local, cap_rows, H, I, act_dt, w_down,
                    w_down_scales, w_dt, y, y_dt, expected_rows, stream);
}

moe_status_t moe_grouped_ffn(const void* xd, const float* xd_scales, const int32_t* offsets,
                             int E_local, int cap_rows, int H, int I, moe_dtype_t act_dt,
                             const void* w_gate, const void* w_up, const void* w_down,
                             const float* w_gate_scales, const float* w_up_scales,
                             const float* w_down_scales, moe_dtype_t w_dt, void* y, moe_dtype_t y_dt,
                             void* ws, size_t ws_bytes, int expected_rows, hipStream_t stream) {
    return grouped_ffn(xd, xd_scales, Rows{offsets, nullptr, 0}, E_local, cap_rows, H, I, act_dt,
                       w_gate, w_up, w_down, w_gate_scales, w_up_scales, w_down_scales, w_dt, y, y_dt,
                       ws, ws_bytes, expected_rows, stream);
}

// masked layout: rows of local expert j are [j*cap_e, j*cap_e + m[j]) of E_local*cap_e
#define MASKED_ROWS()                                                                          \
    REQUIRE(cap_per_expert >= 1, "cap_per_expert must be >= 1 (got %d)", cap_per_expert);     \
    REQUIRE(E_local >= 1 && E_local <= 1024, "E_local must be in [1, 1024] (got %d)", E_local); \
    REQUIRE((long long)E_local * cap_per_expert <= 0x7fffffffLL, "E_local * cap_per_expert must fit in int32")

moe_status_t moe_quant_rows_masked(const void* x, moe_dtype_t x_dt, const int32_t* m, int E_local,
                                   int cap_per_expert, int cols, int8_t* q, float* scales, hipStream_t stream) {
    MASKED_ROWS();
    REQUIRE(m, "null m");
    return quant_rows(x, x_dt, Rows{nullptr, m, cap_per_expert}, E_local, E_local * cap_per_expert, cols, q, scales,
                      stream);
}

moe_status_t moe_ffn_gate_up_masked(const void* xd, const float* xd_scales, const int32_t* m,
                                    int E_local, int cap_per_expert, int H, int I, moe_dtype_t act_dt,
                                    const void* w_gate, const void* w_up, const float* w_gate_scales,
                                    const float* w_up_scales, moe_dtype_t w_dt, void* h,
                                    float* h_scales, int expected_rows, hipStream_t stream) {
    MASKED_ROWS();
    REQUIRE(m, "null m");
    return ffn_gate_up(xd, xd_scales, Rows{nullptr, m, cap_per_expert}, E_local, E_local * cap_per_expert,
                       H, I, act_dt, w_gate, w_up, w_gate_scales, w_up_scales, w_dt, h, h_scales,
                       expected_rows, stream);
}

moe_status_t moe_ffn_down_masked(const void* h, const float* h_scales, const int32_t* m, int E_local,
                                 int cap_per_expert, int H, int I, moe_dtype_t act_dt,
                                 const void* w_down, const float* w_down_scales, moe_dtype_t w_dt,
                                 void* y, moe_dtype_t y_dt, int expected_rows, hipStream_t stream) {
    MASKED_ROWS();
    REQUIRE(m, "null m");
    return ffn_down(h, h_scales, Rows{nullptr, m, cap_per_expert}, E_local, E_local * cap_per_expert,
                    H, I, act_dt, w_down, w_down_scales, w_dt, y, y_dt, expected_rows, stream);
}

moe_status_t moe_grouped_ffn_masked(const void* xd, const float* xd_scales, const int32_t* m,
                                    int E_local, int cap_per_expert, int H, int I, moe_dtype_t act_dt,
                                    const void* w_gate, const void* w_up, const void* w_down,
                                    const float* w_gate_scales, const float* w_up_scales,
                                    const float* w_down_scales, moe_dtype_t w_dt, void* y,
                                    moe_dtype_t y_dt, void* ws, size_t ws_bytes, int expected_rows,
                                    hipStream_t stream) {
    MASKED_ROWS();
    REQUIRE(m, "null m");
    return grouped_ffn(xd, xd_scales, Rows{nullptr, m, cap_per_expert}, E_local,
                       E_local * cap_per_expert, H, I, act_dt, w_gate, w_up, w_down, w_gate_scales,
                       w_up_scales, w_down_scales, w_dt, y, y_dt, ws, ws_bytes, expected_rows, stream);
}

moe_status_t moe_checkpoint_rows(const void* x, moe_dtype_t x_dt, const int32_t* offsets, int E_local, int cap_rows,
                                 int cols, int8_t* q, float* scales, hipStream_t stream) {
    return checkpoint(const_cast<void*>(x), x_dt, offsets, E_local, cap_rows, cols, q, scales, true, stream);
}

moe_status_t moe_checkpoint_values(const int8_t* q, const float* scales, const int32_t* offsets, int E_local,
                                   int cap_rows, int cols, void* out, moe_dtype_t out_dt, hipStream_t stream) {
    return checkpoint(out, out_dt, offsets, E_local, cap_rows, cols, const_cast<int8_t*>(q),
                      const_cast<float*>(scales), false, stream);
}

moe_status_t moe_ffn_gate_up_train(const void* xd, const int32_t* offsets, int E_local, int cap_rows, int H, int I,
                                   moe_dtype_t act_dt, const void* w_gate, const void* w_up, moe_dtype_t w_dt,
                                   void* h, int8_t* gate_q, float* gate_scales, int8_t* up_q, float* up_scales,
                                   int expected_rows, hipStream_t stream) {
    const WType wt = split_w(w_dt);
    moe_status_t s = check_train_dtype(act_dt, wt.dt);
    if (s != MOE_OK) return s;
    s = check_ffn_common(xd, Rows{offsets, nullptr, 0}, E_local, cap_rows, H, I, act_dt, wt.dt);
    if (s != MOE_OK) return s;
    REQUIRE(H <= kTrainCols && I <= kTrainCols, "H and I must be at most %d (got H=%d, I=%d)", kTrainCols, H, I);
    REQUIRE(w_gate && w_up, "null weight pointer");
    REQUIRE((h && gate_q && gate_scales && up_q && up_scales) || cap_rows == 0, "null h or checkpoint pointer");
    REQUIRE(aligned16(w_gate) && aligned16(w_up) && aligned16(h) && aligned16(gate_q) && aligned16(up_q),
            "weights, h and codes must be 16-byte aligned");
    const size_t n = (size_t)cap_rows * I, esz = elem_size(act_dt), w_bytes = (size_t)E_local * I * weight_ld(wt, H) * esz;
    REQUIRE(outputs_apart({{h, n * esz}, {gate_q, n}, {up_q, n}, ckpt_scales(gate_scales, cap_rows, I),
                           ckpt_scales(up_scales, cap_rows, I)},
                          {{xd, (size_t)cap_rows * H * esz}, {w_gate, w_bytes}, {w_up, w_bytes}, ints(offsets, E_local + 1)}),
            "h and the checkpoints must overlap neither each other nor an input");
    auto f = ffn_args(xd, nullptr, Rows{offsets, nullptr, 0}, E_local, cap_rows, H, I, w_gate, w_up, nullptr, nullptr,
                      h, nullptr, expected_rows, wt.dt, weight_ld(wt, H));
    f.gate_q = gate_q;
    f.up_q = up_q;
    f.gate_s = gate_scales;
    f.up_s = up_scales;
    hipError_t e = hipSuccess;
    if (cap_rows > 0) e = act_dt == MOE_F32 ? moeep::launch_ffn_ckpt_f32(f, stream) : moeep::launch_ffn_ckpt_bf16(f, stream);
    return launched(e, "moe_ffn_gate_up_train");
}

moe_status_t moe_swiglu_backward(const void* dh, moe_dtype_t act_dt, const int8_t* gate_q, const float* gate_scales,
                                 const int8_t* up_q, const float* up_scales, int cap_rows, int I,
                                 const int32_t* row_of, const float* topk_w, int B, int K, void* dgate, void* dup,
                                 void* hw, float* dtopk_w, hipStream_t stream) {
    moe_status_t s = check_train_dtype(act_dt, act_dt);
    if (s != MOE_OK) return s;
    REQUIRE(B >= 0 && K >= 1 && K <= 1024, "need B >= 0 and 1 <= K <= 1024");
    REQUIRE((long long)B * K <= 0x7fffffffLL, "B*K must fit in int32");
    REQUIRE(cap_rows >= 0, "cap_rows must be >= 0");
    REQUIRE(I >= 8 && I % 8 == 0 && I <= kTrainCols, "I must be a positive multiple of 8, at most %d (got %d)", kTrainCols, I);
    if (cap_rows > 0) {
        REQUIRE(dh && gate_q && gate_scales && up_q && up_scales && dgate && dup && hw, "null pointer argument");
        REQUIRE(aligned16(dh) && aligned16(gate_q) && aligned16(up_q) && aligned16(dgate) && aligned16(dup) &&
                    aligned16(hw),
                "dh, codes, dgate, dup and hw must be 16-byte aligned");
    }
    if (B > 0) REQUIRE(row_of && topk_w && dtopk_w, "null row_of, topk_w or dtopk_w");
    const size_t n = (size_t)cap_rows * I, nf = n * elem_size(act_dt);
    const Span slots = ints(row_of, (long long)B * K), w{topk_w, slots.bytes}, dw{dtopk_w, slots.bytes};
    const Span gs = ckpt_scales(gate_scales, cap_rows, I), us = ckpt_scales(up_scales, cap_rows, I);
    REQUIRE(outputs_apart({{dgate, nf}, {dup, nf}, {hw, nf}, dw}, {{dh, nf}, {gate_q, n}, {up_q, n}, gs, us, slots}) &&
                outputs_apart({{dgate, nf}, {dup, nf}, {hw, nf}}, {w}) && (dtopk_w == topk_w || apart(dw, w)),
            "outputs must overlap neither each other nor an input (dtopk_w may be topk_w)");
    moeep::SwigluBwdArgs a;
    a.dh = dh;
    a.gate_q = gate_q;
    a.up_q = up_q;
    a.gate_s = gate_scales;
    a.up_s = up_scales;
    a.row_of = row_of;
    a.topk_w = topk_w;
    a.dgate = dgate;
    a.dup = dup;
    a.hw = hw;
    a.dtopk_w = dtopk_w;
    a.cap = cap_rows;
    a.I = I;
    a.slots = (long long)B * K;
    return launched(moeep::launch_swiglu_backward(a, act_dt == MOE_F32, stream), "moe_swiglu_backward");
}

moe_status_t moe_ffn_dgrad(const void* dy, const void* dy2, const int32_t* src_of, int slots_per_token, int src_rows,
                           const int32_t* offsets, int E_local, int cap_rows, int out_dim, int in_dim,
                           moe_dtype_t act_dt, const void* w, const void* w2, moe_dtype_t w_dt, void* dx,
                           int expected_rows, hipStream_t stream) {
    const WType wt = split_w(w_dt);
    moe_status_t s = check_train_dtype(act_dt, wt.dt);
    if (s != MOE_OK) return s;
    s = check_gather(src_of != nullptr, slots_per_token, src_rows);
    if (s != MOE_OK) return s;
    REQUIRE(w && (dx || cap_rows == 0), "null weight or dx pointer");
    s = check_ffn_common(dx, Rows{offsets, nullptr, 0}, E_local, cap_rows, out_dim, in_dim, act_dt, wt.dt, false);
    if (s != MOE_OK) return s;
    REQUIRE(out_dim <= kTrainCols && in_dim <= kTrainCols, "out_dim and in_dim must be at most %d (got %d, %d)", kTrainCols,
            out_dim, in_dim);
    // a buffer of no rows may be null; where src_of names none of no rows, every row of dx is zero
    const bool none = cap_rows == 0 || (src_of && src_rows == 0);
    REQUIRE(dy || none, "null dy");
    REQUIRE((w2 != nullptr) == (dy2 != nullptr) || none, "dy2 and w2 come together");
    REQUIRE(aligned16(dy) && aligned16(dy2) && aligned16(w) && aligned16(w2) && aligned16(dx),
            "dy, weights and dx must be 16-byte aligned");
    const size_t esz = elem_size(act_dt), dy_bytes = (size_t)(src_of ? src_rows : cap_rows) * out_dim * esz,
                 w_bytes = (size_t)E_local * out_dim * weight_ld(wt, in_dim) * esz;
    REQUIRE(outputs_apart({{dx, (size_t)cap_rows * in_dim * esz}},
                          {{dy, dy_bytes}, {dy2, dy_bytes}, {w, w_bytes}, {w2, w_bytes}, ints(src_of, cap_rows),
                           ints(offsets, E_local + 1)}),
            "dx must not overlap an input");
    auto f = ffn_args(dy, nullptr, Rows{offsets, nullptr, 0}, E_local, cap_rows, out_dim, in_dim, w, w2, nullptr,
                      nullptr, dx, nullptr, expected_rows, wt.dt, weight_ld(wt, in_dim));
    f.a2 = w2 ? dy2 : nullptr;
    f.src_of = src_of;
    f.per = src_of ? slots_per_token : 1;
    f.per_div = moeep::divisor_of(f.per);
    f.src_rows = src_rows;
    hipError_t e = hipSuccess;
    if (cap_rows > 0) e = act_dt == MOE_F32 ? moeep::launch_dgrad_f32(f, stream) : moeep::launch_dgrad_bf16(f, stream);
    return launched(e, "moe_ffn_dgrad");
}

moe_status_t moe_ffn_wgrad(const void* dy, const void* dy2, const void* x, moe_dtype_t x_dt, const float* x_scales,
                           const int32_t* src_of, int slots_per_token, int src_rows, moe_gather_t gather,
                           const int32_t* offsets, int E_local, int cap_rows, int out_dim, int in_dim,
                           moe_dtype_t act_dt, const void* base, const void* base2, void* dw, void* dw2,
                           moe_dtype_t dw_dt, int expected_rows, hipStream_t stream) {
    moe_status_t s = check_train_dtype(act_dt, act_dt);
    if (s != MOE_OK) return s;
    if (x_dt != act_dt && x_dt != MOE_CKPT8)
        return fail(MOE_ERR_UNSUPPORTED, "unsupported (act_dt, x_dt) = (%d, %d)", act_dt, x_dt);
    if (!(dw_dt == MOE_F32 || (dw_dt == MOE_BF16 && act_dt == MOE_BF16)))
        return fail(MOE_ERR_UNSUPPORTED, "unsupported (act_dt, dw_dt) = (%d, %d)", act_dt, dw_dt);
    REQUIRE(gather == MOE_GATHER_NONE || gather == MOE_GATHER_X || gather == MOE_GATHER_DY, "unknown gather %d", gather);
    const bool gathers = gather != MOE_GATHER_NONE;
    REQUIRE(!gathers || src_of || cap_rows == 0, "a gathered operand needs src_of");
    s = check_gather(gathers, slots_per_token, src_rows);
    if (s != MOE_OK) return s;
    const int dy_rows = gather == MOE_GATHER_DY ? src_rows : cap_rows, x_rows = gather == MOE_GATHER_X ? src_rows : cap_rows;
    REQUIRE(dw, "null dw");
    s = check_ffn_common(dw, Rows{offsets, nullptr, 0}, E_local, cap_rows, out_dim, in_dim, act_dt, act_dt, false);
    if (s != MOE_OK) return s;
    REQUIRE(out_dim <= kTrainCols && in_dim <= kTrainCols, "out_dim and in_dim must be at most %d (got %d, %d)", kTrainCols,
            out_dim, in_dim);
    const bool none = dy_rows == 0 || x_rows == 0;
    REQUIRE((dy && x) || none, "null dy or x");
    REQUIRE((dw2 != nullptr) == (dy2 != nullptr) || none, "dy2 and dw2 come together");
    REQUIRE(!base2 || dw2, "base2 needs dw2");
    if (x_dt == MOE_CKPT8) REQUIRE(x_scales || none, "a checkpoint x needs its scales");
    REQUIRE(aligned16(dy) && aligned16(dy2) && aligned16(x) && aligned16(base) && aligned16(base2) && aligned16(dw) &&
                aligned16(dw2),
            "dy, x, base and dw must be 16-byte aligned");
    REQUIRE((long long)out_dim * in_dim <= (1ll << 38) / E_local, "dw is too large");
    const size_t dw_bytes = (size_t)E_local * out_dim * in_dim * elem_size(dw_dt);
    const void* const bases[2] = {base, base2};
    void* const dws[2] = {dw, dw2};
    for (int j = 0; j < 2; ++j)
        REQUIRE((bases[j] == dws[j] || apart(bases[j], dw_bytes, dws[j], dw_bytes)) &&
                    apart(bases[j], dw_bytes, dws[1 - j], dw_bytes),
                "a base must be its own dw or lie apart from both");
    const size_t dy_bytes = (size_t)dy_rows * out_dim * elem_size(act_dt),
                 x_bytes = (size_t)x_rows * in_dim * (x_dt == MOE_CKPT8 ? 1 : elem_size(act_dt));
    REQUIRE(outputs_apart({{dw, dw_bytes}, {dw2, dw_bytes}},
                          {{dy, dy_bytes}, {dy2, dy_bytes}, {x, x_bytes},
                           ckpt_scales(x_dt == MOE_CKPT8 ? x_scales : nullptr, x_rows, in_dim),
                           ints(gathers ? src_of : nullptr, cap_rows), ints(offsets, E_local + 1)}),
            "dw and dw2 must overlap neither each other nor an input but their own bases");
    moeep::WgradArgs a;
    a.dy[0] = dy;
    a.dy[1] = dw2 ? dy2 : nullptr;
    a.x = x;
    a.x_scales = x_dt == MOE_CKPT8 ? x_scales : nullptr;
    a.src_of = gathers ? src_of : nullptr;
    a.per = gathers ? slots_per_token : 1;
    a.per_div = moeep::divisor_of(a.per);
    a.src_rows = src_rows;
    a.gather_x = gather == MOE_GATHER_X;
    a.gather_dy = gather == MOE_GATHER_DY;
    a.offsets = offsets;
    a.E_loc = E_local;
    // no rows on one side: sums of none
    a.cap = none ? 0 : cap_rows;
    a.N = out_dim;
    a.M = in_dim;
    a.base[0] = base;
    a.base[1] = base2;
    a.dw[0] = dw;
    a.dw[1] = dw2;
    a.dw_f32 = dw_dt == MOE_F32;
    (void)expected_rows;        // the kernel is chosen by the size of dw
    return launched(act_dt == MOE_F32 ? moeep::launch_wgrad_f32(a, stream) : moeep::launch_wgrad_bf16(a, stream),
                    "moe_ffn_wgrad");
}

moe_status_t moe_route_backward(const void* logits, moe_dtype_t logits_dt, const int32_t* topk_ids,
                                const float* dtopk_w, int B, int E, int K, moe_score_t score, int renorm, float scale,
                                const int32_t* phys_of_logical, int n_shared, float* dlogits, hipStream_t stream) {
    moe_status_t s = check_route_shape(B, E, K);
    if (s != MOE_OK) return s;
    if (logits_dt != MOE_F32 && logits_dt != MOE_BF16)
        return fail(MOE_ERR_UNSUPPORTED, "unsupported logits_dt %d", logits_dt);
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID && score != MOE_SCORE_PICKS)
        return fail(MOE_ERR_UNSUPPORTED, "unsupported score %d", score);
    if (score == MOE_SCORE_PICKS && logits_dt != MOE_F32)
        return fail(MOE_ERR_UNSUPPORTED, "moe_route takes fp32 logits (got logits_dt %d)", logits_dt);
    REQUIRE(std::isfinite(scale), "scale must be finite");
    REQUIRE(score != MOE_SCORE_PICKS || scale == 1.0f, "moe_route's weights have no scale (got %g)", (double)scale);
    REQUIRE(n_shared >= 0 && n_shared <= 1024 - E, "need 0 <= n_shared and E + n_shared <= 1024");
    REQUIRE((long long)B * (K + n_shared) <= 0x7fffffffLL, "B*(K+n_shared) must fit in int32");
    if (B > 0) REQUIRE(logits && topk_ids && dtopk_w && dlogits, "null pointer argument");
    const size_t slots = (size_t)B * (K + n_shared), grid = (size_t)B * E;
    const Span out{dlogits, grid * sizeof(float)};
    // (a token's wave has read a logit before it writes the gradient there)
    REQUIRE(outputs_apart({out}, {ints(topk_ids, slots), {dtopk_w, slots * sizeof(float)}, ints(phys_of_logical, E)}) &&
                ((logits_dt == MOE_F32 && logits == dlogits) || apart(out, Span{logits, grid * elem_size(logits_dt)})),
            "dlogits must not overlap an input (fp32 logits may be its own)");
    moeep::RouteBwdArgs a;
    a.logits = logits;
    a.ids = topk_ids;
    a.dw = dtopk_w;
    a.map = phys_of_logical;
    a.dlogits = dlogits;
    a.scale = scale;
    a.B = B;
    a.E = E;
    a.K = K;
    a.Kt = K + n_shared;
    a.score = score;
    a.bf16 = logits_dt == MOE_BF16;
    a.renorm = renorm != 0;
    return launched(moeep::launch_route_backward(a, stream), "moe_route_backward");
}

moe_status_t moe_combine(const void* y, moe_dtype_t y_dt, int cap_rows, const int32_t* row_of,
                         const float* topk_w, int B, int K, int H, void* out, moe_dtype_t out_dt,
                         hipStream_t stream) {
    REQUIRE(B >= 0 && K >= 1 && K <= 1024, "need B >= 0 and 1 <= K <= 1024");
    REQUIRE((long long)B * K <= 0x7fffffffLL, "B*K must fit in int32");
    REQUIRE(H >= 8 && H % 8 == 0, "H must be a positive multiple of 8 (got %d)", H);
    REQUIRE(cap_rows >= 0, "cap_rows must be >= 0");
    int kind;
    if (y_dt == MOE_F32 && out_dt == MOE_F32) kind = 0;
    else if (y_dt == MOE_BF16 && out_dt == MOE_BF16) kind = 1;
    else if (y_dt == MOE_BF16 && out_dt == MOE_F32) kind = 2;
    else return fail(MOE_ERR_UNSUPPORTED, "unsupported combine (y_dt, out_dt) = (%d, %d)", y_dt, out_dt);
    if (B > 0) {
        REQUIRE((y || cap_rows == 0) && row_of && topk_w && out, "null pointer argument");
        REQUIRE(aligned16(y) && aligned16(out), "y and out must be 16-byte aligned");
    }
    return launched(moeep::launch_combine(y, kind, row_of, topk_w, B, K, H, out, cap_rows, stream),
                    "moe_combine");
}

}  // extern "C"
