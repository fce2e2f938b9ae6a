// C entry points of the 8-bit operators (include/rankmixer.h, "8-bit operands
// and checkpoints"): argument checks, workspace layout, launches.
#include <nvtx3/nvToolsExt.h>

#include <mutex>
#include <new>
#include <unordered_map>

#include "../../include/rankmixer.h"
#include "rm_fp8.h"
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
#define RM_CHECK_CUDA(expr, what)                          \
    do {                                                   \
        cudaError_t _e = (expr);                           \
        if (_e != cudaSuccess) return cuda_fail(_e, what); \
    } while (0)
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
#define RM_LAUNCH(kind, what, ...)                               \
    do {                                                         \
        const Range _r("rm:fp8_" #kind);                         \
        RM_CHECK_CUDA(launch_fp8_##kind(__VA_ARGS__), what);     \
    } while (0)
#define RM_CHECK(expr)                        \
    do {                                      \
        rm_status _s = (expr);                \
        if (_s != RM_OK) return _s;           \
    } while (0)

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1u)) == 0; }
long long up(long long v, long long m) { return (v + m - 1) / m * m; }
bool known(rm_dtype d) { return d == RM_F32 || d == RM_BF16; }
cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

Fp8View view(const rm_fp8_tensor& t) {
    return Fp8View{(uint8_t*)t.codes, t.scales, t.ld, t.lds, t.format == RM_E5M2};
}

// rows are limited so that row and block numbers of every kernel fit 32-bit grids
constexpr long long kMaxRows = 1ll << 31;
// ... and every other size so that rounding it up to whole tiles does not overflow
constexpr int kMaxSize = 0x7fffffff - 511;
// Summed lengths.  The tensor cores' accumulator truncates as it adds, about a unit
// in the last place an instruction (32 products, or 16 of the weight gradient), so
// sums that stay in it are held to lengths at which terms of one sign lose less than
// 2^-9, below bf16's own rounding: K of the products, and B of bf16 gradients (2^21
// samples lost 1.2%, 2^17 0.05%).  Float32 gradients join sums of 2048 samples with
// rounding to nearest; their B only keeps a tile's time well inside the waits' bound.
constexpr int kMaxK = 1 << 19;
constexpr int kMaxBatchBf16 = 1 << 17;
constexpr int kMaxBatch = 1 << 27;

constexpr unsigned long long kWaitTimeoutNs = 2000000000ull;    // bound of every device-side wait

// The error word of the tensor-core kernels, one per device that loads the library;
// what rm_fp8_sync_status took from it, and a flag that nothing sets (the test hook's).
__device__ int g_fp8_error, g_fp8_taken, g_fp8_unset;

// Read and cleared at once: an error latched meanwhile is in this word or the next one.
__global__ void take_error_kernel() { g_fp8_taken = atomicExch(&g_fp8_error, 0); }

// The word does not tell whose call ran out, so every stream that asks is told of every
// error once: how many there were, the latest, and how many each stream (by its
// identifier, which is not reused) has been told of.
struct Reported {
    std::mutex mu;
    unsigned long long count = 0;
    int last = 0;
    std::unordered_map<unsigned long long, unsigned long long> seen;
};
constexpr int kMaxDevices = 64;

// SM count and error word of the current device, looked up once per device.
rm_status device_info(Fp8Device* out) {
    static std::mutex mu;
    static Fp8Device known_devices[kMaxDevices];
    int d = 0;
    RM_CHECK_CUDA(cudaGetDevice(&d), "cudaGetDevice");
    if (d < 0 || d >= kMaxDevices) return fail(RM_ERR_UNSUPPORTED, "device %d", d);
    std::lock_guard<std::mutex> lk(mu);
    Fp8Device& k = known_devices[d];
    if (!k.err) {
        int n = 0;
        void* p = nullptr;
        RM_CHECK_CUDA(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d), "SM count");
        RM_CHECK_CUDA(cudaGetSymbolAddress(&p, g_fp8_error), "error word");
        k.num_sms = n;
        k.timeout_ns = kWaitTimeoutNs;
        k.err = (int*)p;
    }
    *out = k;
    return RM_OK;
}

rm_status check_tensor(const rm_fp8_tensor* t, int cols, const char* name, bool e4m3_only) {
    if (!t) return fail(RM_ERR_INVALID_ARG, "%s is NULL", name);
    if (!t->codes || !t->scales) return fail(RM_ERR_INVALID_ARG, "%s has NULL codes or scales", name);
    if (t->format != RM_E4M3 && t->format != RM_E5M2) return fail(RM_ERR_INVALID_ARG, "%s: unknown format", name);
    if (e4m3_only && t->format != RM_E4M3) return fail(RM_ERR_UNSUPPORTED, "%s must be e4m3", name);
    if (!aligned(t->codes, 16) || !aligned(t->scales, 4))
        return fail(RM_ERR_INVALID_ARG, "%s: codes must be 16-byte and scales 4-byte aligned", name);
    if (t->ld < cols || t->ld % 16 != 0)
        return fail(RM_ERR_INVALID_ARG, "%s: ld (%lld) must be a multiple of 16 and hold %d columns", name, t->ld, cols);
    if (t->lds < (cols + kFp8Block - 1) / kFp8Block || t->lds % 4 != 0)
        return fail(RM_ERR_INVALID_ARG, "%s: lds (%lld) must be a multiple of 4 and hold a byte per %d columns of %d",
                    name, t->lds, kFp8Block, cols);
    return RM_OK;
}

rm_status check_sizes(int B, int T, int K, int N) {
    if (B < 1 || T < 1 || K < 1 || N < 1) return fail(RM_ERR_INVALID_ARG, "sizes must be positive");
    if (B > kMaxSize || K > kMaxSize || N > kMaxSize) return fail(RM_ERR_INVALID_ARG, "sizes are at most 2^31 - 512");
    if (T > 65535) return fail(RM_ERR_INVALID_ARG, "T (%d) is at most 65535", T);
    if ((long long)B * T >= kMaxRows) return fail(RM_ERR_INVALID_ARG, "B T (%d x %d) must be below 2^31", B, T);
    return RM_OK;
}

rm_status check_rows(long long rows, int cols) {
    if (rows < 1 || rows >= kMaxRows || cols < 1 || cols > kMaxSize)
        return fail(RM_ERR_INVALID_ARG, "rows must be in [1, 2^31), cols in [1, 2^31 - 512]");
    return RM_OK;
}

rm_status check_batch(int B, rm_dtype grads) {
    if (B > kMaxBatch) return fail(RM_ERR_UNSUPPORTED, "B (%d) is at most 2^27", B);
    if (grads == RM_BF16 && B > kMaxBatchBf16)
        return fail(RM_ERR_UNSUPPORTED, "B (%d) is at most 2^17 for bf16 gradients (float32 ones take more)", B);
    return RM_OK;
}

rm_status check_ffn(const rm_fp8_pffn* p) {
    if (!p) return fail(RM_ERR_INVALID_ARG, "p is NULL");
    RM_CHECK(check_sizes(1, p->T, p->D, p->F));
    if (p->D % 16 != 0 || p->F % 16 != 0)
        return fail(RM_ERR_UNSUPPORTED, "D (%d) and F (%d) must be multiples of 16", p->D, p->F);
    if (p->D > kMaxK || p->F > kMaxK)
        return fail(RM_ERR_UNSUPPORTED, "D (%d) and F (%d) are at most 2^19", p->D, p->F);
    RM_CHECK(check_tensor(&p->W1, p->F, "W1", true));
    RM_CHECK(check_tensor(&p->W2, p->D, "W2", true));
    if (!p->b1 || !p->b2) return fail(RM_ERR_INVALID_ARG, "b1 / b2 is NULL");
    if (!aligned(p->b1, 16) || !aligned(p->b2, 16))
        return fail(RM_ERR_INVALID_ARG, "b1 and b2 must be 16-byte aligned");
    return RM_OK;
}

rm_status check_kept(const rm_fp8_kept* k, const rm_fp8_pffn* p) {
    RM_CHECK(check_tensor(&k->x, p->D, "kept x", true));
    RM_CHECK(check_tensor(&k->u, p->F, "kept u", true));
    return check_tensor(&k->a, p->F, "kept a", true);
}

// Workspace pieces, each 256-byte aligned from a 16-byte aligned start.
struct Carver {
    char* base;
    long long used = 0;
    void* take(long long bytes) {
        void* p = base ? base + used : nullptr;
        used += up(bytes, 256);
        return p;
    }
    rm_fp8_tensor tensor(long long rows, int cols) {
        rm_fp8_tensor t;
        t.ld = up(cols, 16);
        t.lds = up((cols + kFp8Block - 1) / kFp8Block, 4);
        t.codes = take(rows * t.ld);
        t.scales = (unsigned char*)take(rows * t.lds);
        t.format = RM_E4M3;
        return t;
    }
};

struct ForwardWork {
    rm_fp8_kept kept;
    long long bytes;
};
ForwardWork forward_work(const rm_fp8_pffn* p, int B, const rm_fp8_kept* keep, bool train, void* base) {
    Carver c{(char*)base};
    const long long rows = (long long)B * p->T;
    ForwardWork w{};
    if (keep)
        w.kept = *keep;
    else if (!train) {
        w.kept.x = c.tensor(rows, p->D);
        w.kept.a = c.tensor(rows, p->F);
    }
    w.bytes = c.used;
    return w;
}

struct BackwardWork {
    rm_fp8_tensor dv, du;
    void *dv16, *du16;
    long long bytes;
};
BackwardWork backward_work(const rm_fp8_pffn* p, int B, void* base) {
    Carver c{(char*)base};
    const long long rows = (long long)B * p->T;
    BackwardWork w{};
    w.dv = c.tensor(rows, p->D);
    w.du = c.tensor(rows, p->F);
    w.dv16 = c.take(rows * p->D * 2);
    w.du16 = c.take(rows * p->F * 2);
    w.bytes = c.used;
    return w;
}

rm_status check_work(const void* work, long long have, long long need) {
    if (need > 0 && !work) return fail(RM_ERR_INVALID_ARG, "work is NULL");
    if (!aligned(work, 16)) return fail(RM_ERR_INVALID_ARG, "work must be 16-byte aligned");
    if (have < need) return fail(RM_ERR_INVALID_ARG, "work_bytes (%lld) is below the %lld needed", have, need);
    return RM_OK;
}

Fp8Product product(rm_dtype dtype, const rm_fp8_tensor& x, const rm_fp8_tensor& w, bool trans, const float* bias,
                   void* y, int B, int T, int K, int N) {
    Fp8Product p{};
    p.epi = dtype == RM_F32 ? FP8_OUT_F32 : FP8_OUT_BF16;
    p.x = view(x), p.w = view(w), p.trans = trans, p.bias = bias, p.y = y;
    p.B = B, p.T = T, p.K = K, p.N = N;
    return p;
}

}  // namespace

namespace rm {
int fp8_device(Fp8Device* out) { return device_info(out); }
}  // namespace rm

rm_status rm_fp8_quantize(const void* X, rm_dtype dtype, long long rows, int cols, long long ldx,
                          const rm_fp8_tensor* out, void* stream) {
    if (!X) return fail(RM_ERR_INVALID_ARG, "X is NULL");
    if (!known(dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    RM_CHECK(check_rows(rows, cols));
    if (ldx < cols) return fail(RM_ERR_INVALID_ARG, "ldx (%lld) is below cols (%d)", ldx, cols);
    if (!aligned(X, dtype == RM_F32 ? 4 : 2)) return fail(RM_ERR_INVALID_ARG, "X must be aligned to its elements");
    RM_CHECK(check_tensor(out, cols, "out", false));
    RM_LAUNCH(quantize, "quantize", dtype == RM_F32, X, rows, cols, ldx, view(*out), nullptr, as_stream(stream));
    return RM_OK;
}

rm_status rm_fp8_quantize_weight(const void* W, rm_dtype dtype, int T, int K, int N, const rm_fp8_tensor* out,
                                 void* stream) {
    if (!W) return fail(RM_ERR_INVALID_ARG, "W is NULL");
    if (!known(dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    RM_CHECK(check_sizes(1, T, K, N));
    if ((K + kFp8Block - 1) / kFp8Block > 65535) return fail(RM_ERR_INVALID_ARG, "K (%d) is too large", K);
    if (!aligned(W, dtype == RM_F32 ? 4 : 2)) return fail(RM_ERR_INVALID_ARG, "W must be aligned to its elements");
    RM_CHECK(check_tensor(out, N, "out", true));
    RM_LAUNCH(quantize_weight, "quantize weight", dtype == RM_F32, W, T, K, N, view(*out), as_stream(stream));
    return RM_OK;
}

rm_status rm_fp8_dequantize(const rm_fp8_tensor* in, long long rows, int cols, void* Y, rm_dtype dtype, long long ldy,
                            void* stream) {
    if (!Y) return fail(RM_ERR_INVALID_ARG, "Y is NULL");
    if (!known(dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    RM_CHECK(check_rows(rows, cols));
    if (ldy < cols) return fail(RM_ERR_INVALID_ARG, "ldy (%lld) is below cols (%d)", ldy, cols);
    if (!aligned(Y, dtype == RM_F32 ? 4 : 2)) return fail(RM_ERR_INVALID_ARG, "Y must be aligned to its elements");
    RM_CHECK(check_tensor(in, cols, "in", false));
    RM_LAUNCH(dequantize, "dequantize", view(*in), rows, cols, Y, dtype == RM_F32, ldy, as_stream(stream));
    return RM_OK;
}

rm_status rm_fp8_matmul(const rm_fp8_tensor* x, const rm_fp8_tensor* W, const float* bias, void* Y, rm_dtype dtype,
                        int B, int T, int K, int N, int transpose_w, void* stream) {
    if (!Y) return fail(RM_ERR_INVALID_ARG, "Y is NULL");
    if (!known(dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    RM_CHECK(check_sizes(B, T, K, N));
    if (K > kMaxK) return fail(RM_ERR_UNSUPPORTED, "K (%d) is at most 2^19", K);
    RM_CHECK(check_tensor(x, K, "x", false));
    RM_CHECK(check_tensor(W, transpose_w ? K : N, "W", true));
    if (!aligned(Y, 16) || (bias && !aligned(bias, 16)))
        return fail(RM_ERR_INVALID_ARG, "Y and bias must be 16-byte aligned");
    Fp8Device dev;
    RM_CHECK(device_info(&dev));
    RM_LAUNCH(product, "8-bit product", product(dtype, *x, *W, transpose_w != 0, bias, Y, B, T, K, N), dev, as_stream(stream));
    return RM_OK;
}

rm_status rm_fp8_wgrad(const rm_fp8_tensor* x, const void* dY, void* dW, void* db, rm_dtype dtype, int B, int T, int K,
                       int N, void* stream) {
    if (!dY || !dW) return fail(RM_ERR_INVALID_ARG, "dY / dW is NULL");
    if (!known(dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    RM_CHECK(check_sizes(B, T, K, N));
    if (N % 8 != 0) return fail(RM_ERR_UNSUPPORTED, "N (%d) must be a multiple of 8", N);
    RM_CHECK(check_batch(B, dtype));
    RM_CHECK(check_tensor(x, K, "x", true));
    if (!aligned(dY, 16) || !aligned(dW, 16) || (db && !aligned(db, 16)))
        return fail(RM_ERR_INVALID_ARG, "dY, dW and db must be 16-byte aligned");
    const cudaStream_t s = as_stream(stream);
    Fp8Device dev;
    RM_CHECK(device_info(&dev));
    RM_LAUNCH(wgrad, "weight gradient", view(*x), dY, dW, db, dtype == RM_F32, B, T, K, N, dev, s);
    return RM_OK;
}

rm_status rm_fp8_pffn_workspace(const rm_fp8_pffn* p, int B, rm_fp8_pass pass, long long* bytes) {
    if (!bytes) return fail(RM_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    RM_CHECK(check_ffn(p));
    RM_CHECK(check_sizes(B, p->T, p->D, p->F));
    if (pass == RM_FP8_SERVE || pass == RM_FP8_TRAIN)
        *bytes = forward_work(p, B, nullptr, pass == RM_FP8_TRAIN, nullptr).bytes;
    else if (pass == RM_FP8_BACKWARD)
        *bytes = backward_work(p, B, nullptr).bytes;
    else
        return fail(RM_ERR_INVALID_ARG, "unknown pass");
    return RM_OK;
}

rm_status rm_fp8_pffn_forward(const rm_fp8_pffn* p, const void* X, rm_dtype x_dtype, void* V, rm_dtype v_dtype,
                              const rm_fp8_kept* keep, int B, void* work, long long work_bytes, void* stream) {
    RM_CHECK(check_ffn(p));
    if (!X || !V) return fail(RM_ERR_INVALID_ARG, "X / V is NULL");
    if (!known(x_dtype) || !known(v_dtype)) return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    if (!aligned(X, 16) || !aligned(V, 16)) return fail(RM_ERR_INVALID_ARG, "X and V must be 16-byte aligned");
    RM_CHECK(check_sizes(B, p->T, p->D, p->F));
    if (keep) RM_CHECK(check_kept(keep, p));
    const ForwardWork w = forward_work(p, B, keep, keep != nullptr, work);
    RM_CHECK(check_work(work, work_bytes, w.bytes));
    const int T = p->T, D = p->D, F = p->F;
    const long long rows = (long long)B * T;
    const cudaStream_t s = as_stream(stream);
    Fp8Device dev;
    RM_CHECK(device_info(&dev));
    RM_LAUNCH(quantize, "quantize", x_dtype == RM_F32, X, rows, D, D, view(w.kept.x), nullptr, s);
    Fp8Product g = product(RM_BF16, w.kept.x, p->W1, false, p->b1, nullptr, B, T, D, F);
    g.epi = FP8_GELU;
    g.follows = true;
    g.o0 = view(w.kept.a);
    if (keep) g.o1 = view(w.kept.u);
    RM_LAUNCH(product, "8-bit layer 1", g, dev, s);
    g = product(v_dtype, w.kept.a, p->W2, false, p->b2, V, B, T, F, D);
    g.follows = true;
    RM_LAUNCH(product, "8-bit layer 2", g, dev, s);
    return RM_OK;
}

rm_status rm_fp8_pffn_backward(const rm_fp8_pffn* p, const void* dV, rm_dtype dv_dtype, const rm_fp8_kept* kept,
                               void* dX, rm_dtype dx_dtype, const rm_fp8_grads* grads, int B, void* work,
                               long long work_bytes, void* stream) {
    RM_CHECK(check_ffn(p));
    if (!dV || !kept || !grads) return fail(RM_ERR_INVALID_ARG, "dV / kept / grads is NULL");
    if (!known(dv_dtype) || (dX && !known(dx_dtype)) || !known(grads->dtype))
        return fail(RM_ERR_INVALID_ARG, "unknown dtype");
    if (!grads->dW1 || !grads->db1 || !grads->dW2 || !grads->db2)
        return fail(RM_ERR_INVALID_ARG, "a gradient buffer is NULL");
    for (const void* q : {dV, (const void*)dX, (const void*)grads->dW1, (const void*)grads->db1, (const void*)grads->dW2,
                          (const void*)grads->db2})
        if (!aligned(q, 16)) return fail(RM_ERR_INVALID_ARG, "dV, dX and the gradients must be 16-byte aligned");
    RM_CHECK(check_sizes(B, p->T, p->D, p->F));
    RM_CHECK(check_batch(B, grads->dtype));
    RM_CHECK(check_kept(kept, p));
    const BackwardWork w = backward_work(p, B, work);
    RM_CHECK(check_work(work, work_bytes, w.bytes));
    const int T = p->T, D = p->D, F = p->F;
    const long long rows = (long long)B * T;
    const bool f32 = dv_dtype == RM_F32, g32 = grads->dtype == RM_F32;
    const cudaStream_t s = as_stream(stream);
    Fp8Device dev;
    RM_CHECK(device_info(&dev));
    const void* dv16 = f32 ? w.dv16 : dV;
    RM_LAUNCH(quantize, "quantize dV", f32, dV, rows, D, D, view(w.dv), f32 ? w.dv16 : nullptr, s);
    Fp8Product g = product(RM_BF16, w.dv, p->W2, true, nullptr, w.du16, B, T, D, F);
    g.epi = FP8_DGELU;
    g.follows = true;
    g.o0 = view(w.du);
    g.o1 = view(kept->u);
    RM_LAUNCH(product, "dU", g, dev, s);
    if (dX) {
        g = product(dx_dtype, w.du, p->W1, true, nullptr, dX, B, T, F, D);
        g.follows = true;
        RM_LAUNCH(product, "dX", g, dev, s);
    }
    RM_LAUNCH(wgrad, "dW2", view(kept->a), dv16, grads->dW2, grads->db2, g32, B, T, F, D, dev, s);
    RM_LAUNCH(wgrad, "dW1", view(kept->x), w.du16, grads->dW1, grads->db1, g32, B, T, D, F, dev, s);
    return RM_OK;
}

rm_status rm_fp8_sync_status(void* stream) {
    const cudaStream_t s = as_stream(stream);
    cudaError_t e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "rm_fp8_sync_status");
    Fp8Device dev;
    RM_CHECK(device_info(&dev));
    int d = 0, v = 0;
    unsigned long long id = 0;
    RM_CHECK_CUDA(cudaGetDevice(&d), "cudaGetDevice");
    RM_CHECK_CUDA(cudaStreamGetId(s, &id), "cudaStreamGetId");
    static Reported reported[kMaxDevices];
    Reported& r = reported[d];
    std::lock_guard<std::mutex> lk(r.mu);
    take_error_kernel<<<1, 1, 0, s>>>();
    RM_CHECK_CUDA(cudaGetLastError(), "error word");
    RM_CHECK_CUDA(cudaMemcpyFromSymbolAsync(&v, g_fp8_taken, sizeof v, 0, cudaMemcpyDeviceToHost, s), "error word");
    RM_CHECK_CUDA(cudaStreamSynchronize(s), "error word");
    if (v != 0) ++r.count, r.last = v;
    try {
        unsigned long long& seen = r.seen[id];
        if (seen == r.count) return RM_OK;
        seen = r.count;
    } catch (const std::bad_alloc&) {
        return fail(RM_ERR_OOM, "rm_fp8_sync_status");
    }
    return r.last == kDevErrTimeout ? fail(RM_ERR_TIMEOUT, "a device-side wait of an 8-bit or 4-bit operator ran out")
                                    : fail(RM_ERR_DEVICE, "device error %d in an 8-bit or 4-bit operator", r.last);
}

rm_status rm_debug_fp8_wait_timeout(int timeout_us, void* stream) {
    if (timeout_us < 1 || timeout_us > 10000000) return fail(RM_ERR_INVALID_ARG, "timeout_us out of range");
    Fp8Device dev;
    RM_CHECK(device_info(&dev));
    void* flag = nullptr;
    RM_CHECK_CUDA(cudaGetSymbolAddress(&flag, g_fp8_unset), "flag");
    RM_CHECK_CUDA(launch_debug_wait((const int*)flag, dev.err, (unsigned long long)timeout_us * 1000ull, as_stream(stream)),
                  "debug wait");
    return RM_OK;
}
