// C entry points of the 4-bit operators and of the experts' rows
// (include/rankmixer.h, "4-bit operands" and "Rows by expert"): argument checks,
// workspace layout, launches.
#include <nvtx3/nvToolsExt.h>

#include "../../include/rankmixer.h"
#include "rm_fp4.h"
#include "rm_internal.h"

using namespace rm;

namespace {

template <typename... A>
rm_status fail(rm_status st, const char* fmt, A... a) {
    set_last_error(fmt, a...);
    return st;
}
rm_status cuda_fail(cudaError_t e, const char* what) {
    if (e == cudaErrorInvalidValue)
        if (const char* cond = take_debug_bounds())
            return fail(RM_ERR_INVALID_ARG, "%s: bounds check failed: %s", what, cond);
    if (e == cudaErrorNotSupported) return fail(RM_ERR_UNSUPPORTED, "%s: shape not supported by this kernel", what);
    return fail(e == cudaErrorMemoryAllocation ? RM_ERR_OOM : RM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}
// A launch, in an NVTX range of its kind's name where these are on (RM_NVTX).
struct Range {
    const bool on = nvtx_on();
    explicit Range(const char* name) {
        if (on) nvtxRangePushA(name);
    }
    ~Range() {
        if (on) nvtxRangePop();
    }
};
#define RM_LAUNCH(kind, what, ...)                          \
    do {                                                    \
        const Range _r("rm:" #kind);                        \
        cudaError_t _e = launch_##kind(__VA_ARGS__);        \
        if (_e != cudaSuccess) return cuda_fail(_e, what);  \
    } while (0)
#define RM_CHECK(expr)                        \
    do {                                      \
        rm_status _s = (rm_status)(expr);     \
        if (_s != RM_OK) return _s;           \
    } while (0)

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1u)) == 0; }
long long up(long long v, long long m) { return (v + m - 1) / m * m; }
bool known(rm_dtype d) { return d == RM_F32 || d == RM_BF16; }
unsigned size_of(rm_dtype d) { return d == RM_F32 ? 4u : 2u; }
cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
Fp4View view(const rm_fp4_tensor& t) { return Fp4View{(uint8_t*)t.codes, t.scales, t.ld, t.lds}; }

// Limits as of the 8-bit calls: rows and blocks in 32-bit grids, sizes that can be
// rounded up to whole tiles, sums whose truncation stays below 2^-9.
constexpr long long kMaxRows = 1ll << 31;
constexpr int kMaxSize = 0x7fffffff - 511;
constexpr int kMaxK = 1 << 19;
constexpr int kMaxGroups = 65535;

rm_status check_tensor(const rm_fp4_tensor* t, int cols, const char* name, bool weight) {
    if (!t) return fail(RM_ERR_INVALID_ARG, "%s is NULL", name);
    if (!t->codes || !t->scales) return fail(RM_ERR_INVALID_ARG, "%s has NULL codes or scales", name);
    if (!aligned(t->codes, 16) || !aligned(t->scales, 16))
        return fail(RM_ERR_INVALID_ARG, "%s: codes and scales must be 16-byte aligned", name);
    if (t->ld % 16 != 0 || t->ld < 16 * fp4_blocks(cols))
        return fail(RM_ERR_INVALID_ARG, "%s: ld (%lld) must be a multiple of 16 and hold %d columns", name, t->ld, cols);
    if (weight ? t->lds != fp4_weight_quads(cols) : t->lds % 16 != 0 || t->lds < fp4_blocks(cols))
        return weight ? fail(RM_ERR_INVALID_ARG, "%s: lds (%lld) must be 2 ceil(%d / 256)", name, t->lds, cols)
                      : fail(RM_ERR_INVALID_ARG, "%s: lds (%lld) must be a multiple of 16 and hold a byte per 32 of %d columns",
                             name, t->lds, cols);
    return RM_OK;
}
rm_status check_rows(long long rows, int cols) {
    if (rows < 1 || rows >= kMaxRows || cols < 1 || cols > kMaxSize)
        return fail(RM_ERR_INVALID_ARG, "rows must be in [1, 2^31), cols in [1, 2^31 - 512]");
    return RM_OK;
}
// groups of at most B rows, products over K with N columns
rm_status check_product(int B, int G, int K, int N) {
    if (B < 1 || G < 1 || K < 1 || N < 1) return fail(RM_ERR_INVALID_ARG, "sizes must be positive");
    if (B > kMaxSize || K > kMaxSize || N > kMaxSize) return fail(RM_ERR_INVALID_ARG, "sizes are at most 2^31 - 512");
    if (G > kMaxGroups) return fail(RM_ERR_INVALID_ARG, "T, or T E (%d), is at most 65535", G);
    if (K > kMaxK) return fail(RM_ERR_UNSUPPORTED, "K (%d) is at most 2^19", K);
    return RM_OK;
}
rm_status check_batch(int B, int T, int E) {
    if (B < 1 || T < 1 || E < 1) return fail(RM_ERR_INVALID_ARG, "sizes must be positive");
    if ((long long)T * E > kMaxGroups) return fail(RM_ERR_INVALID_ARG, "T E (%d x %d) is at most 65535", T, E);
    if (B > kMaxSize || (long long)B * T * E >= kMaxRows)
        return fail(RM_ERR_INVALID_ARG, "B T E (%d x %d x %d) must be below 2^31", B, T, E);
    return RM_OK;
}
rm_status check_sorted(const rm_expert_rows* r) {
    if (!r) return fail(RM_ERR_INVALID_ARG, "rows is NULL");
    if (!r->offsets || !r->source || !r->slot || !r->tiles)
        return fail(RM_ERR_INVALID_ARG, "rows: offsets / source / slot / tiles is NULL");
    if (!aligned(r->offsets, 4) || !aligned(r->source, 4) || !aligned(r->slot, 4) || !aligned(r->tiles, 16))
        return fail(RM_ERR_INVALID_ARG, "rows: tiles must be 16-byte aligned, the rest to their elements");
    return check_batch(r->B, r->T, r->E);
}
// sorted rows [n][D] of a pass over X or V [B][T][D]
rm_status check_pass(const rm_expert_rows* r, long long n, int D) {
    RM_CHECK(check_sorted(r));
    if (D < 1 || D > kMaxSize) return fail(RM_ERR_INVALID_ARG, "D must be in [1, 2^31 - 512]");
    if (n < 0 || n >= kMaxRows) return fail(RM_ERR_INVALID_ARG, "n must be in [0, 2^31)");
    return RM_OK;
}
ExpertRows sorted(const rm_expert_rows& r) {
    return ExpertRows{r.offsets, r.source, r.slot, reinterpret_cast<int4*>(r.tiles), r.B, r.T, r.E};
}

rm_status check_ffn(const rm_fp4_tensor& W1, const rm_fp4_tensor& W2, const float* b1, const float* b2, int G, int D, int F) {
    RM_CHECK(check_product(1, G, D, F));
    if (D % 32 != 0 || F % 32 != 0) return fail(RM_ERR_UNSUPPORTED, "D (%d) and F (%d) must be multiples of 32", D, F);
    if (F > kMaxK) return fail(RM_ERR_UNSUPPORTED, "F (%d) is at most 2^19", F);
    RM_CHECK(check_tensor(&W1, D, "W1", true));
    RM_CHECK(check_tensor(&W2, F, "W2", true));
    if (!b1 || !b2) return fail(RM_ERR_INVALID_ARG, "b1 / b2 is NULL");
    if (!aligned(b1, 16) || !aligned(b2, 16)) return fail(RM_ERR_INVALID_ARG, "b1 and b2 must be 16-byte aligned");
    return RM_OK;
}
rm_status check_pffn(const rm_fp4_pffn* p, int B) {
    if (!p) return fail(RM_ERR_INVALID_ARG, "p is NULL");
    RM_CHECK(check_ffn(p->W1, p->W2, p->b1, p->b2, p->T, p->D, p->F));
    RM_CHECK(check_product(B, p->T, p->D, p->F));
    if ((long long)B * p->T >= kMaxRows) return fail(RM_ERR_INVALID_ARG, "B T (%d x %d) must be below 2^31", B, p->T);
    return RM_OK;
}
rm_status check_moe(const rm_fp4_moe* p, int B) {
    if (!p) return fail(RM_ERR_INVALID_ARG, "p is NULL");
    RM_CHECK(check_batch(B, p->T, p->E));
    return check_ffn(p->W1, p->W2, p->b1, p->b2, p->T * p->E, p->D, p->F);
}
rm_status check_work(const void* work, long long have, long long need) {
    if (need > 0 && !work) return fail(RM_ERR_INVALID_ARG, "work is NULL");
    if (!aligned(work, 16)) return fail(RM_ERR_INVALID_ARG, "work must be 16-byte aligned");
    if (have < need) return fail(RM_ERR_INVALID_ARG, "work_bytes (%lld) is below the %lld needed", have, need);
    return RM_OK;
}

// Workspace pieces, each 256-byte aligned from the start.
struct Carver {
    char* base;
    long long used = 0;
    void* take(long long bytes) {
        void* p = base ? base + used : nullptr;
        used += up(bytes, 256);
        return p;
    }
    Fp4View rows(long long n, int cols) {
        Fp4View v;
        v.ld = 16 * fp4_blocks(cols), v.lds = up(fp4_blocks(cols), 16);
        v.codes = (uint8_t*)take(n * v.ld);
        v.scales = (uint8_t*)take(n * v.lds);
        return v;
    }
};
struct PffnWork {
    Fp4View x, a;
    long long bytes;
};
PffnWork pffn_work(const rm_fp4_pffn* p, int B, void* base) {
    Carver c{(char*)base};
    PffnWork w{};
    w.x = c.rows((long long)B * p->T, p->D);
    w.a = c.rows((long long)B * p->T, p->F);
    w.bytes = c.used;
    return w;
}
// The experts' outputs wait for their gates in float32 at every size: in bf16 above some
// size a sample's precision would hang on how many others it is served with (1024 samples
// of T = 32, E = 8, D = 1536, F = 2048, a quarter open: 409-417 us, error in norm 0.0017; in
// bf16 354 and 0.0024).
struct MoeWork {
    ExpertRows rows;
    int* sort;
    Fp4View x, a;
    float* y;
    long long n, bytes;
};
MoeWork moe_work(const rm_fp4_moe* p, int B, void* base) {
    Carver c{(char*)base};
    MoeWork w{};
    const long long TE = (long long)p->T * p->E;
    w.n = B * TE;
    w.rows.B = B, w.rows.T = p->T, w.rows.E = p->E;
    w.rows.offsets = (int*)c.take(4 * (TE + 1));
    w.rows.source = (int*)c.take(4 * w.n);
    w.rows.slot = (int*)c.take(4 * w.n);
    w.rows.tiles = (int4*)c.take(16 * (1 + TE * ((B + kExpertTile - 1) / kExpertTile)));
    w.sort = (int*)c.take(4 * expert_sort_work(B, p->T, p->E));
    w.x = c.rows(w.n, p->D);
    w.a = c.rows(w.n, p->F);
    w.y = (float*)c.take(4 * w.n * p->D);
    w.bytes = c.used;
    return w;
}

Fp4Product product(rm_dtype dtype, const Fp4View& x, const Fp4View& w, const float* bias, void* y, int B, int G, int K,
                   int N) {
    Fp4Product p{};
    p.epi = dtype == RM_F32 ? FP4_OUT_F32 : FP4_OUT_BF16;
    p.x = x, p.w = w, p.bias = bias, p.y = y;
    p.B = B, p.G = G, p.K = K, p.N = N;
    p.n = (long long)B * G;
    return p;
}

}  // namespace

rm_status rm_fp4_quantize(const void* X, rm_dtype dtype, long long rows, int cols, long long ldx,
                          const rm_fp4_tensor* out, void* stream) {
    if (!X) return fail(RM_ERR_INVALID_ARG, "X is NULL");
    if (!known(dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    RM_CHECK(check_rows(rows, cols));
    if (ldx < cols) return fail(RM_ERR_INVALID_ARG, "ldx (%lld) is below cols (%d)", ldx, cols);
    if (!aligned(X, size_of(dtype))) return fail(RM_ERR_INVALID_ARG, "X must be aligned to its elements");
    RM_CHECK(check_tensor(out, cols, "out", false));
    RM_LAUNCH(fp4_quantize, "quantize", dtype == RM_F32, X, rows, cols, ldx, view(*out), as_stream(stream));
    return RM_OK;
}

rm_status rm_fp4_quantize_weight(const void* W, rm_dtype dtype, int G, int K, int N, const rm_fp4_tensor* out,
                                 void* stream) {
    if (!W) return fail(RM_ERR_INVALID_ARG, "W is NULL");
    if (!known(dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    RM_CHECK(check_product(1, G, K, N));
    if (!aligned(W, size_of(dtype))) return fail(RM_ERR_INVALID_ARG, "W must be aligned to its elements");
    RM_CHECK(check_tensor(out, K, "out", true));
    RM_LAUNCH(fp4_quantize_weight, "quantize weight", dtype == RM_F32, W, G, K, N, view(*out), as_stream(stream));
    return RM_OK;
}

rm_status rm_fp4_dequantize(const rm_fp4_tensor* in, long long rows, int cols, void* Y, rm_dtype dtype, long long ldy,
                            void* stream) {
    if (!Y) return fail(RM_ERR_INVALID_ARG, "Y is NULL");
    if (!known(dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    RM_CHECK(check_rows(rows, cols));
    if (ldy < cols) return fail(RM_ERR_INVALID_ARG, "ldy (%lld) is below cols (%d)", ldy, cols);
    if (!aligned(Y, size_of(dtype))) return fail(RM_ERR_INVALID_ARG, "Y must be aligned to its elements");
    RM_CHECK(check_tensor(in, cols, "in", false));
    RM_LAUNCH(fp4_dequantize, "dequantize", view(*in), rows, cols, Y, dtype == RM_F32, ldy, as_stream(stream));
    return RM_OK;
}

rm_status rm_fp4_matmul(const rm_fp4_tensor* x, const rm_fp4_tensor* W, const float* bias, void* Y, rm_dtype dtype,
                        int B, int T, int K, int N, void* stream) {
    if (!Y) return fail(RM_ERR_INVALID_ARG, "Y is NULL");
    if (!known(dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    RM_CHECK(check_product(B, T, K, N));
    if ((long long)B * T >= kMaxRows) return fail(RM_ERR_INVALID_ARG, "B T (%d x %d) must be below 2^31", B, T);
    RM_CHECK(check_tensor(x, K, "x", false));
    RM_CHECK(check_tensor(W, K, "W", true));
    if (!aligned(Y, 16) || (bias && !aligned(bias, 16)))
        return fail(RM_ERR_INVALID_ARG, "Y and bias must be 16-byte aligned");
    Fp8Device dev;
    RM_CHECK(fp8_device(&dev));
    RM_LAUNCH(fp4_product, "4-bit product", product(dtype, view(*x), view(*W), bias, Y, B, T, K, N), dev,
              as_stream(stream));
    return RM_OK;
}

rm_status rm_fp4_pffn_workspace(const rm_fp4_pffn* p, int B, long long* bytes) {
    if (!bytes) return fail(RM_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    RM_CHECK(check_pffn(p, B));
    *bytes = pffn_work(p, B, nullptr).bytes;
    return RM_OK;
}

rm_status rm_fp4_pffn_forward(const rm_fp4_pffn* p, const void* X, rm_dtype x_dtype, void* V, rm_dtype v_dtype, int B,
                              void* work, long long work_bytes, void* stream) {
    RM_CHECK(check_pffn(p, B));
    if (!X || !V) return fail(RM_ERR_INVALID_ARG, "X / V is NULL");
    if (!known(x_dtype) || !known(v_dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    if (!aligned(X, 16) || !aligned(V, 16)) return fail(RM_ERR_INVALID_ARG, "X and V must be 16-byte aligned");
    const PffnWork w = pffn_work(p, B, work);
    RM_CHECK(check_work(work, work_bytes, w.bytes));
    const int T = p->T, D = p->D, F = p->F;
    const cudaStream_t s = as_stream(stream);
    Fp8Device dev;
    RM_CHECK(fp8_device(&dev));
    RM_LAUNCH(fp4_quantize, "quantize", x_dtype == RM_F32, X, (long long)B * T, D, D, w.x, s);
    Fp4Product g = product(RM_BF16, w.x, view(p->W1), p->b1, nullptr, B, T, D, F);
    g.epi = FP4_GELU;
    g.o = w.a;
    g.follows = true;
    RM_LAUNCH(fp4_product, "4-bit layer 1", g, dev, s);
    g = product(v_dtype, w.a, view(p->W2), p->b2, V, B, T, F, D);
    g.follows = true;
    RM_LAUNCH(fp4_product, "4-bit layer 2", g, dev, s);
    return RM_OK;
}

rm_status rm_expert_sort_workspace(int B, int T, int E, long long* bytes) {
    if (!bytes) return fail(RM_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    RM_CHECK(check_batch(B, T, E));
    *bytes = 4 * expert_sort_work(B, T, E);
    return RM_OK;
}

rm_status rm_expert_sort(const float* G, const rm_expert_rows* rows, void* work, long long work_bytes, void* stream) {
    if (!G) return fail(RM_ERR_INVALID_ARG, "G is NULL");
    if (!aligned(G, 4)) return fail(RM_ERR_INVALID_ARG, "G must be aligned to its elements");
    RM_CHECK(check_sorted(rows));
    RM_CHECK(check_work(work, work_bytes, 4 * expert_sort_work(rows->B, rows->T, rows->E)));
    RM_LAUNCH(expert_sort, "sort by expert", G, sorted(*rows), (int*)work, as_stream(stream));
    return RM_OK;
}

rm_status rm_expert_gather(const void* X, rm_dtype dtype, const rm_expert_rows* rows, void* Xs, long long n, int D,
                           void* stream) {
    RM_CHECK(check_pass(rows, n, D));
    if (!X || (n > 0 && !Xs)) return fail(RM_ERR_INVALID_ARG, "X / Xs is NULL");
    if (!known(dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    if (!aligned(X, size_of(dtype)) || !aligned(Xs, size_of(dtype)))
        return fail(RM_ERR_INVALID_ARG, "X and Xs must be aligned to their elements");
    if (n == 0) return RM_OK;
    RM_LAUNCH(expert_gather, "gather", X, dtype == RM_F32, sorted(*rows), Xs, n, D, as_stream(stream));
    return RM_OK;
}

rm_status rm_fp4_expert_gather(const void* X, rm_dtype dtype, const rm_expert_rows* rows, const rm_fp4_tensor* out,
                               long long n, int D, void* stream) {
    RM_CHECK(check_pass(rows, n, D));
    if (!X) return fail(RM_ERR_INVALID_ARG, "X is NULL");
    if (!known(dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    if (!aligned(X, size_of(dtype))) return fail(RM_ERR_INVALID_ARG, "X must be aligned to its elements");
    if (n == 0) return RM_OK;
    RM_CHECK(check_tensor(out, D, "out", false));
    RM_LAUNCH(fp4_expert_gather, "gather", X, dtype == RM_F32, sorted(*rows), view(*out), n, D, as_stream(stream));
    return RM_OK;
}

rm_status rm_expert_combine(const void* Y, rm_dtype y_dtype, const rm_expert_rows* rows, const float* G, void* V,
                            rm_dtype v_dtype, long long n, int D, void* stream) {
    RM_CHECK(check_pass(rows, n, D));
    if ((n > 0 && !Y) || !V) return fail(RM_ERR_INVALID_ARG, "Y / V is NULL");
    if (!known(y_dtype) || !known(v_dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    if (!aligned(Y, size_of(y_dtype)) || !aligned(V, size_of(v_dtype)) || !aligned(G, 4))
        return fail(RM_ERR_INVALID_ARG, "Y, G and V must be aligned to their elements");
    RM_LAUNCH(expert_combine, "combine", Y, y_dtype == RM_F32, sorted(*rows), G, V, v_dtype == RM_F32, n, D,
              as_stream(stream));
    return RM_OK;
}

rm_status rm_expert_combine_backward(const void* dV, const void* Y, rm_dtype dtype, const rm_expert_rows* rows,
                                     const float* G, void* dY, float* dG, long long n, int D, void* stream) {
    RM_CHECK(check_pass(rows, n, D));
    if (!dV || !G || !dG || (n > 0 && (!Y || !dY))) return fail(RM_ERR_INVALID_ARG, "dV / Y / G / dY / dG is NULL");
    if (!known(dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    for (const void* q : {dV, Y, (const void*)dY})
        if (!aligned(q, size_of(dtype))) return fail(RM_ERR_INVALID_ARG, "dV, Y and dY must be aligned to their elements");
    if (!aligned(G, 4) || !aligned(dG, 4)) return fail(RM_ERR_INVALID_ARG, "G and dG must be aligned to their elements");
    RM_LAUNCH(expert_combine_backward, "combine backward", dV, Y, dtype == RM_F32, sorted(*rows), G, dY, dG, n, D,
              as_stream(stream));
    return RM_OK;
}

rm_status rm_fp4_expert_matmul(const rm_fp4_tensor* x, const rm_fp4_tensor* W, const rm_expert_rows* rows,
                               const float* bias, void* Y, rm_dtype dtype, long long n, int K, int N, void* stream) {
    RM_CHECK(check_pass(rows, n, 1));
    if (!known(dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    RM_CHECK(check_product(rows->B, rows->T * rows->E, K, N));
    RM_CHECK(check_tensor(W, K, "W", true));
    if (!aligned(Y, 16) || (bias && !aligned(bias, 16)))
        return fail(RM_ERR_INVALID_ARG, "Y and bias must be 16-byte aligned");
    if (n == 0) return RM_OK;
    if (!Y) return fail(RM_ERR_INVALID_ARG, "Y is NULL");
    RM_CHECK(check_tensor(x, K, "x", false));
    Fp8Device dev;
    RM_CHECK(fp8_device(&dev));
    Fp4Product g = product(dtype, view(*x), view(*W), bias, Y, rows->B, rows->T * rows->E, K, N);
    g.tiles = reinterpret_cast<const int4*>(rows->tiles);
    g.n = n;
    RM_LAUNCH(fp4_product, "experts' product", g, dev, as_stream(stream));
    return RM_OK;
}

rm_status rm_fp4_moe_workspace(const rm_fp4_moe* p, int B, long long* bytes) {
    if (!bytes) return fail(RM_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    RM_CHECK(check_moe(p, B));
    *bytes = moe_work(p, B, nullptr).bytes;
    return RM_OK;
}

rm_status rm_fp4_moe_forward(const rm_fp4_moe* p, const void* X, rm_dtype x_dtype, const float* G, void* V,
                             rm_dtype v_dtype, int B, void* work, long long work_bytes, void* stream) {
    RM_CHECK(check_moe(p, B));
    if (!X || !G || !V) return fail(RM_ERR_INVALID_ARG, "X / G / V is NULL");
    if (!known(x_dtype) || !known(v_dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    if (!aligned(X, 16) || !aligned(V, 16) || !aligned(G, 4))
        return fail(RM_ERR_INVALID_ARG, "X and V must be 16-byte aligned, G to its elements");
    const MoeWork w = moe_work(p, B, work);
    RM_CHECK(check_work(work, work_bytes, w.bytes));
    const int D = p->D, F = p->F, groups = p->T * p->E;
    const cudaStream_t s = as_stream(stream);
    Fp8Device dev;
    RM_CHECK(fp8_device(&dev));
    RM_LAUNCH(expert_sort, "sort by expert", G, w.rows, w.sort, s);
    RM_LAUNCH(fp4_expert_gather, "gather", X, x_dtype == RM_F32, w.rows, w.x, w.n, D, s);
    Fp4Product g = product(RM_BF16, w.x, view(p->W1), p->b1, nullptr, B, groups, D, F);
    g.epi = FP4_GELU;
    g.o = w.a;
    g.tiles = w.rows.tiles;
    g.n = w.n;
    g.follows = true;
    RM_LAUNCH(fp4_product, "experts' layer 1", g, dev, s);
    g = product(RM_F32, w.a, view(p->W2), p->b2, w.y, B, groups, F, D);
    g.tiles = w.rows.tiles;
    g.n = w.n;
    g.follows = true;
    RM_LAUNCH(fp4_product, "experts' layer 2", g, dev, s);
    RM_LAUNCH(expert_combine, "combine", w.y, true, w.rows, G, V, v_dtype == RM_F32, w.n, D, s);
    return RM_OK;
}
