// The C ABI: argument validation (before any CUDA call, so refusals need no GPU), the device check,
// error reporting and dispatch to the kernel families.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>

#include "../../include/q4gemv.h"
#include "block.h"
#include "kv.h"
#include "launch.h"

namespace q4 {

namespace {

thread_local std::string g_last_error;

int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return code;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int cuda_fail(const char* what, cudaError_t e) {
    if (e == cudaErrorNotSupported)
        return fail(Q4_EUNSUPPORTED, "%s: the staged input does not fit in shared memory next to the weight rings",
                    what);
    return fail(Q4_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

// The device check: the library carries sm_103a code only.
int check_device(const char* what, DeviceInfo* di) {
    cudaError_t e = current_device_info(di);
    if (e != cudaSuccess) return cuda_fail(what, e);
    if (di->major != 10 || di->minor != 3)
        return fail(Q4_EUNSUPPORTED, "%s: device is sm_%d%d, this library is built for sm_103a", what, di->major,
                    di->minor);
    return Q4_OK;
}

int check_eps(const char* what, float eps) {
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(Q4_EINVAL, "%s: eps must be finite and >= 0", what);
    return Q4_OK;
}

int check_q4_weights(const char* what, const uint8_t* qs, const uint16_t* d, int N, int K) {
    if (!qs || !d) return fail(Q4_EINVAL, "%s: null weight pointer", what);
    if (N <= 0) return fail(Q4_EINVAL, "%s: N must be >= 1 (got %d)", what, N);
    if (K <= 0 || K % 32 != 0) return fail(Q4_EINVAL, "%s: K must be a positive multiple of 32 (got %d)", what, K);
    if (!aligned(qs, 16)) return fail(Q4_EALIGN, "%s: qs must be 16-byte aligned", what);
    if (!aligned(d, 2)) return fail(Q4_EALIGN, "%s: d must be 2-byte aligned", what);
    return Q4_OK;
}

int check_q4k_weights(const char* what, const uint8_t* w, int N, int K) {
    if (!w) return fail(Q4_EINVAL, "%s: null weight pointer", what);
    if (N <= 0) return fail(Q4_EINVAL, "%s: N must be >= 1 (got %d)", what, N);
    if (K <= 0 || K % 256 != 0) return fail(Q4_EINVAL, "%s: K must be a positive multiple of 256 (got %d)", what, K);
    if (!aligned(w, 16)) return fail(Q4_EALIGN, "%s: weights must be 16-byte aligned", what);
    return Q4_OK;
}

int check_out(const char* what, const float* y, uintptr_t a = 4) {
    if (!y) return fail(Q4_EINVAL, "%s: null output pointer", what);
    if (!aligned(y, a)) return fail(Q4_EALIGN, "%s: output must be %d-byte aligned", what, (int)a);
    return Q4_OK;
}

int check_vec(const char* what, const char* name, const float* v) {
    if (!v) return fail(Q4_EINVAL, "%s: null %s", what, name);
    if (!aligned(v, 16)) return fail(Q4_EALIGN, "%s: %s must be 16-byte aligned", what, name);
    return Q4_OK;
}

#define Q4_TRY(expr)            \
    do {                        \
        int rc_ = (expr);       \
        if (rc_ != Q4_OK) return rc_; \
    } while (0)

int finish(const char* what, cudaError_t e) {
    if (e != cudaSuccess) return cuda_fail(what, e);
    g_last_error.clear();
    return Q4_OK;
}

}  // namespace

namespace {
std::atomic<int> g_launch_overlap{0};
std::atomic<long long> g_wait_limit{4000000000LL};
}  // namespace

bool launch_overlap() { return g_launch_overlap.load(std::memory_order_relaxed) != 0; }

long long wait_limit_cycles() { return g_wait_limit.load(std::memory_order_relaxed); }

// The fault word every kernel family ORs its kFault* bits into (one per device that loads the library).
static __device__ unsigned g_faults;

unsigned* device_fault_word(int device) {
    static unsigned* ptrs[64] = {};
    static std::mutex mu;
    if (device < 0 || device >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!ptrs[device]) {
        unsigned* p = nullptr;
        if (cudaGetSymbolAddress((void**)&p, g_faults) != cudaSuccess) return nullptr;
        ptrs[device] = p;
    }
    return ptrs[device];
}

static cudaError_t read_and_clear_faults(unsigned* out) {
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_faults, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_faults, &zero, sizeof(unsigned));
    return e;
}

cudaError_t current_device_info(DeviceInfo* out) {
    static DeviceInfo cache[64];
    static std::mutex mu;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev].device != dev) {
        DeviceInfo di;
        di.device = dev;
        if ((e = cudaDeviceGetAttribute(&di.sm_count, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&di.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) !=
            cudaSuccess)
            return e;
        if ((e = cudaDeviceGetAttribute(&di.major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&di.minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess) return e;
        cache[dev] = di;
    }
    *out = cache[dev];
    return cudaSuccess;
}

}  // namespace q4

using namespace q4;

extern "C" {

int q4_gemv(float* y, const uint8_t* qs, const uint16_t* d, const float* x, int N, int K, q4_stream_t stream) {
    const char* what = "q4_gemv";
    Q4_TRY(check_out(what, y));
    Q4_TRY(check_q4_weights(what, qs, d, N, K));
    Q4_TRY(check_vec(what, "x", x));
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_q4_gemv(y, qs, d, x, 1, N, K, (cudaStream_t)stream));
}

int q4_gemv_batched(float* Y, const uint8_t* qs, const uint16_t* d, const float* X, int M, int N, int K,
                    q4_stream_t stream) {
    const char* what = "q4_gemv_batched";
    Q4_TRY(check_out(what, Y));
    Q4_TRY(check_q4_weights(what, qs, d, N, K));
    Q4_TRY(check_vec(what, "X", X));
    if (M < 1 || M > 16) return fail(Q4_EINVAL, "%s: M=%d outside 1..16 (refused, not clamped)", what, M);
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_q4_gemv(Y, qs, d, X, M, N, K, (cudaStream_t)stream));
}

int fused_rmsnorm_q4k_gemv(float* y, const uint8_t* w, const float* x, const float* gamma, float eps, int N, int K,
                           q4_stream_t stream) {
    const char* what = "fused_rmsnorm_q4k_gemv";
    Q4_TRY(check_out(what, y));
    Q4_TRY(check_q4k_weights(what, w, N, K));
    Q4_TRY(check_vec(what, "x", x));
    Q4_TRY(check_vec(what, "gamma", gamma));
    Q4_TRY(check_eps(what, eps));
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_q4k_gemv(y, nullptr, w, nullptr, x, gamma, eps, N, K, false, (cudaStream_t)stream));
}

int q4k_gemv_batched(float* Y, const uint8_t* w, const float* X, int M, int N, int K, q4_stream_t stream) {
    const char* what = "q4k_gemv_batched";
    Q4_TRY(check_out(what, Y));
    Q4_TRY(check_q4k_weights(what, w, N, K));
    Q4_TRY(check_vec(what, "X", X));
    if (M < 1 || M > 8) return fail(Q4_EINVAL, "%s: M=%d outside 1..8 (refused, not clamped)", what, M);
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_q4k_gemv_batched(Y, w, X, M, N, K, (cudaStream_t)stream));
}

int fused_gateup_q4k_gemv(float* y_gate, float* y_up, const uint8_t* w_gate, const uint8_t* w_up, const float* x,
                          const float* gamma, float eps, int N, int K, q4_stream_t stream) {
    const char* what = "fused_gateup_q4k_gemv";
    Q4_TRY(check_out(what, y_gate));
    Q4_TRY(check_out(what, y_up));
    Q4_TRY(check_q4k_weights(what, w_gate, N, K));
    Q4_TRY(check_q4k_weights(what, w_up, N, K));
    Q4_TRY(check_vec(what, "x", x));
    if (gamma) Q4_TRY(check_vec(what, "gamma", gamma));
    Q4_TRY(check_eps(what, eps));
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_q4k_gemv(y_gate, y_up, w_gate, w_up, x, gamma, eps, N, K, false, (cudaStream_t)stream));
}

static int check_moe(const char* what, const float* y_gate, const float* y_up, const uint8_t* qs_gate,
                     const uint16_t* d_gate, const uint8_t* qs_up, const uint16_t* d_up, const int32_t* ids, int T,
                     int topk, int E, int N, int K) {
    Q4_TRY(check_out(what, y_gate));
    Q4_TRY(check_out(what, y_up));
    if (E <= 0) return fail(Q4_EINVAL, "%s: E must be >= 1 (got %d)", what, E);
    if ((long long)E * N > 0x7fffffffLL) return fail(Q4_EINVAL, "%s: E*N exceeds 2^31-1 rows", what);
    Q4_TRY(check_q4_weights(what, qs_gate, d_gate, N, K));
    Q4_TRY(check_q4_weights(what, qs_up, d_up, N, K));
    if (!ids) return fail(Q4_EINVAL, "%s: null expert_ids", what);
    if (!aligned(ids, 4)) return fail(Q4_EALIGN, "%s: expert_ids must be 4-byte aligned", what);
    if (T <= 0 || topk <= 0) return fail(Q4_EINVAL, "%s: T and topk must be >= 1", what);
    if (topk > E) return fail(Q4_EINVAL, "%s: topk=%d exceeds E=%d", what, topk, E);
    if ((long long)T * topk > 512) return fail(Q4_EINVAL, "%s: T*topk=%lld exceeds 512", what, (long long)T * topk);
    return Q4_OK;
}

int moe_q4_gemv(float* y_gate, float* y_up, const uint8_t* qs_gate, const uint16_t* d_gate, const uint8_t* qs_up,
                const uint16_t* d_up, const float* x, const int32_t* expert_ids, int T, int topk, int E, int N, int K,
                int32_t* dev_status, q4_stream_t stream) {
    const char* what = "moe_q4_gemv";
    Q4_TRY(check_moe(what, y_gate, y_up, qs_gate, d_gate, qs_up, d_up, expert_ids, T, topk, E, N, K));
    Q4_TRY(check_vec(what, "x", x));
    if (dev_status && !aligned(dev_status, 4)) return fail(Q4_EALIGN, "%s: dev_status must be 4-byte aligned", what);
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_moe_q4_gemv(y_gate, y_up, qs_gate, d_gate, qs_up, d_up, x, expert_ids, T, topk, E, N,
                                           K, dev_status, false, false, (cudaStream_t)stream));
}

int fused_gateup_swiglu_q4k_gemv(float* y, const uint8_t* w_gate, const uint8_t* w_up, const float* x,
                                 const float* gamma, float eps, int N, int K, q4_stream_t stream) {
    const char* what = "fused_gateup_swiglu_q4k_gemv";
    Q4_TRY(check_out(what, y));
    Q4_TRY(check_q4k_weights(what, w_gate, N, K));
    Q4_TRY(check_q4k_weights(what, w_up, N, K));
    Q4_TRY(check_vec(what, "x", x));
    if (gamma) Q4_TRY(check_vec(what, "gamma", gamma));
    Q4_TRY(check_eps(what, eps));
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_q4k_gemv(y, nullptr, w_gate, w_up, x, gamma, eps, N, K, true, (cudaStream_t)stream));
}

int moe_q4_swiglu_gemv(float* y, const uint8_t* qs_gate, const uint16_t* d_gate, const uint8_t* qs_up,
                       const uint16_t* d_up, const float* x, const int32_t* expert_ids, int T, int topk, int E, int N,
                       int K, int32_t* dev_status, q4_stream_t stream) {
    const char* what = "moe_q4_swiglu_gemv";
    Q4_TRY(check_moe(what, y, y, qs_gate, d_gate, qs_up, d_up, expert_ids, T, topk, E, N, K));
    Q4_TRY(check_vec(what, "x", x));
    if (dev_status && !aligned(dev_status, 4)) return fail(Q4_EALIGN, "%s: dev_status must be 4-byte aligned", what);
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_moe_q4_gemv(y, nullptr, qs_gate, d_gate, qs_up, d_up, x, expert_ids, T, topk, E, N, K,
                                           dev_status, false, true, (cudaStream_t)stream));
}

int moe_router_q4(int32_t* expert_ids, float* expert_weights, float* logits, const uint8_t* qs, const uint16_t* d,
                  const float* x, int T, int E, int K, int topk, int normalize, q4_stream_t stream) {
    const char* what = "moe_router_q4";
    if (!expert_ids || !expert_weights) return fail(Q4_EINVAL, "%s: null output pointer", what);
    if (!aligned(expert_ids, 4) || !aligned(expert_weights, 4) || (logits && !aligned(logits, 4)))
        return fail(Q4_EALIGN, "%s: outputs must be 4-byte aligned", what);
    if (E <= 0 || E > 4096) return fail(Q4_EINVAL, "%s: E must be in 1..4096 (got %d)", what, E);
    Q4_TRY(check_q4_weights(what, qs, d, E, K));
    Q4_TRY(check_vec(what, "x", x));
    if (T <= 0) return fail(Q4_EINVAL, "%s: T must be >= 1 (got %d)", what, T);
    if (topk <= 0 || topk > E) return fail(Q4_EINVAL, "%s: topk must be in 1..E (got %d, E=%d)", what, topk, E);
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_moe_router(expert_ids, expert_weights, logits, qs, d, x, T, E, K, topk, normalize != 0,
                                          (cudaStream_t)stream));
}

int q4_pure_read(float* sink, const uint8_t* qs, const uint16_t* d, int N, int K, q4_stream_t stream) {
    const char* what = "q4_pure_read";
    Q4_TRY(check_out(what, sink));
    Q4_TRY(check_q4_weights(what, qs, d, N, K));
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_q4_pure_read(sink, qs, d, N, K, (cudaStream_t)stream));
}

int q4k_pure_read(float* sink, const uint8_t* w, int N, int K, q4_stream_t stream) {
    const char* what = "q4k_pure_read";
    Q4_TRY(check_out(what, sink));
    Q4_TRY(check_q4k_weights(what, w, N, K));
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_q4k_pure_read(sink, w, N, K, (cudaStream_t)stream));
}

int moe_q4_pure_read(float* sink_gate, float* sink_up, const uint8_t* qs_gate, const uint16_t* d_gate,
                     const uint8_t* qs_up, const uint16_t* d_up, const int32_t* expert_ids, int T, int topk, int E,
                     int N, int K, int32_t* dev_status, q4_stream_t stream) {
    const char* what = "moe_q4_pure_read";
    Q4_TRY(check_moe(what, sink_gate, sink_up, qs_gate, d_gate, qs_up, d_up, expert_ids, T, topk, E, N, K));
    if (dev_status && !aligned(dev_status, 4)) return fail(Q4_EALIGN, "%s: dev_status must be 4-byte aligned", what);
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_moe_q4_gemv(sink_gate, sink_up, qs_gate, d_gate, qs_up, d_up, nullptr, expert_ids, T,
                                           topk, E, N, K, dev_status, true, false, (cudaStream_t)stream));
}

int q4_fma_ceiling(float* sink, int sink_len, long long fmas, float mul, float add, long long* fmas_done,
                   q4_stream_t stream) {
    const char* what = "q4_fma_ceiling";
    Q4_TRY(check_out(what, sink));
    if (fmas <= 0) return fail(Q4_EINVAL, "%s: fmas must be >= 1 (got %lld)", what, fmas);
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    if (sink_len < di.sm_count)
        return fail(Q4_EINVAL, "%s: sink holds %d floats, the launch writes one per SM (%d)", what, sink_len,
                    di.sm_count);
    const long long per = fma_ceiling_fmas_per_iter(di.sm_count);
    const long long iters = (fmas + per - 1) / per;
    if (fmas_done) *fmas_done = iters * per;
    return finish(what, launch_fma_ceiling(sink, iters, mul, add, di.sm_count, (cudaStream_t)stream));
}

int q4_dequant(float* W, const uint8_t* qs, const uint16_t* d, int N, int K, q4_stream_t stream) {
    const char* what = "q4_dequant";
    Q4_TRY(check_out(what, W, 16));
    Q4_TRY(check_q4_weights(what, qs, d, N, K));
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_q4_dequant(W, qs, d, N, K, (cudaStream_t)stream));
}

int q4k_dequant(float* W, const uint8_t* w, int N, int K, q4_stream_t stream) {
    const char* what = "q4k_dequant";
    Q4_TRY(check_out(what, W, 16));
    Q4_TRY(check_q4k_weights(what, w, N, K));
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    return finish(what, launch_q4k_dequant(W, w, N, K, (cudaStream_t)stream));
}

static size_t dtype_bytes(int dtype) { return dtype == Q4_F32 ? 4 : 2; }

static int check_dtype(const char* what, int dtype) {
    if (dtype != Q4_F32 && dtype != Q4_F16 && dtype != Q4_BF16)
        return fail(Q4_EINVAL, "%s: dtype must be Q4_F32, Q4_F16 or Q4_BF16 (got %d)", what, dtype);
    return Q4_OK;
}

// Rows of activations: [tokens] of `width` elements, `stride` elements apart, every row 16-byte aligned.
static int check_rows(const char* what, const char* name, const void* p, long long stride, long long width, int dtype) {
    if (!p) return fail(Q4_EINVAL, "%s: null %s", what, name);
    if (stride < width)
        return fail(Q4_EINVAL, "%s: token stride of %s is %lld, below its row of %lld elements", what, name, stride, width);
    if (!aligned(p, 16) || (stride * (long long)dtype_bytes(dtype)) % 16 != 0)
        return fail(Q4_EALIGN, "%s: every row of %s must be 16-byte aligned", what, name);
    return Q4_OK;
}

static int check_heads(const char* what, int Hkv, int D) {
    if (Hkv <= 0) return fail(Q4_EINVAL, "%s: the number of key heads must be >= 1 (got %d)", what, Hkv);
    if (D <= 0 || D % 32 != 0 || D > 256)
        return fail(Q4_EINVAL, "%s: the head size must be a multiple of 32 up to 256 (got %d)", what, D);
    if ((long long)Hkv * D > (1 << 20)) return fail(Q4_EINVAL, "%s: key heads * head size exceeds 2^20", what);
    return Q4_OK;
}

static int check_cache(const char* what, const kv4_cache* c) {
    if (!c) return fail(Q4_EINVAL, "%s: null cache", what);
    if (!c->k_qs || !c->k_d || !c->v_qs || !c->v_d) return fail(Q4_EINVAL, "%s: null cache pointer", what);
    Q4_TRY(check_heads(what, c->num_kv_heads, c->head_dim));
    if (c->num_pages <= 0) return fail(Q4_EINVAL, "%s: num_pages must be >= 1 (got %d)", what, c->num_pages);
    if (c->page_size <= 0 || (c->page_size & (c->page_size - 1)) != 0)
        return fail(Q4_EINVAL, "%s: page_size must be a power of two (got %d)", what, c->page_size);
    if ((long long)c->num_pages * c->page_size * c->num_kv_heads > 0x7fffffffLL)
        return fail(Q4_EINVAL, "%s: the cache exceeds 2^31-1 rows", what);
    if (!aligned(c->k_qs, 16) || !aligned(c->v_qs, 16))
        return fail(Q4_EALIGN, "%s: k_qs and v_qs must be 16-byte aligned", what);
    if (!aligned(c->k_d, 16) || !aligned(c->v_d, 16))
        return fail(Q4_EALIGN, "%s: k_d and v_d must be 16-byte aligned", what);
    return Q4_OK;
}

static int log2_of(int n) {  // of a power of two
    int l = 0;
    while ((1 << l) < n) ++l;
    return l;
}

static int check_index(const char* what, const char* name, const int32_t* p) {
    if (!p) return fail(Q4_EINVAL, "%s: null %s", what, name);
    if (!aligned(p, 4)) return fail(Q4_EALIGN, "%s: %s must be 4-byte aligned", what, name);
    return Q4_OK;
}

// The device check, and the fault word that the kernels record in.
static int check_device_faults(const char* what, DeviceInfo* di, unsigned** fault) {
    Q4_TRY(check_device(what, di));
    *fault = device_fault_word(di->device);
    if (!*fault) return fail(Q4_ECUDA, "%s: the device's fault word cannot be resolved", what);
    return Q4_OK;
}

int qk_norm_rope(void* q_out, void* k_out, const void* q, const void* k, const float* q_gamma, const float* k_gamma,
                 float eps, const float* cos_sin, const int32_t* positions, int T, int Hq, int Hkv, int D, int rot_dim,
                 int max_pos, int interleaved, long long q_stride, long long k_stride, long long q_out_stride,
                 long long k_out_stride, int dtype, q4_stream_t stream) {
    const char* what = "qk_norm_rope";
    if (T <= 0) return fail(Q4_EINVAL, "%s: T must be >= 1 (got %d)", what, T);
    Q4_TRY(check_dtype(what, dtype));
    Q4_TRY(check_heads(what, Hkv, D));
    if (Hq <= 0 || Hq > 65535 || Hkv > 65535) return fail(Q4_EINVAL, "%s: 1 to 65535 heads are taken", what);
    if ((long long)T * (Hq + Hkv) > 0x7fffffffLL) return fail(Q4_EINVAL, "%s: T * heads exceeds 2^31-1", what);
    Q4_TRY(check_rows(what, "q", q, q_stride, (long long)Hq * D, dtype));
    Q4_TRY(check_rows(what, "k", k, k_stride, (long long)Hkv * D, dtype));
    Q4_TRY(check_rows(what, "q_out", q_out, q_out_stride, (long long)Hq * D, dtype));
    Q4_TRY(check_rows(what, "k_out", k_out, k_out_stride, (long long)Hkv * D, dtype));
    if (q_gamma) Q4_TRY(check_vec(what, "q_gamma", q_gamma));
    if (k_gamma) Q4_TRY(check_vec(what, "k_gamma", k_gamma));
    Q4_TRY(check_eps(what, eps));
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0)
        return fail(Q4_EINVAL, "%s: rot_dim must be a multiple of 16 up to the head size (got %d)", what, rot_dim);
    if (rot_dim > 0) {
        if (max_pos <= 0) return fail(Q4_EINVAL, "%s: max_pos must be >= 1 (got %d)", what, max_pos);
        Q4_TRY(check_vec(what, "cos_sin", cos_sin));
        Q4_TRY(check_index(what, "positions", positions));
    }
    DeviceInfo di;
    RopeArgs a = {q_out, k_out, q, k, q_gamma, k_gamma, cos_sin, positions, eps, T, Hq, Hkv, D, rot_dim, max_pos,
                  interleaved != 0, q_stride, k_stride, q_out_stride, k_out_stride, nullptr, 0};
    Q4_TRY(check_device_faults(what, &di, &a.fault));
    a.sm_count = di.sm_count;
    return finish(what, launch_qk_norm_rope(a, dtype, (cudaStream_t)stream));
}

int kv4_write(const kv4_cache* cache, const void* k, const void* v, const int32_t* slots, int T, long long k_stride,
              long long v_stride, int dtype, q4_stream_t stream) {
    const char* what = "kv4_write";
    Q4_TRY(check_cache(what, cache));
    if (T <= 0 || T > (1 << 30)) return fail(Q4_EINVAL, "%s: T must be in 1..2^30 (got %d)", what, T);
    Q4_TRY(check_dtype(what, dtype));
    const long long width = (long long)cache->num_kv_heads * cache->head_dim;
    Q4_TRY(check_rows(what, "k", k, k_stride, width, dtype));
    Q4_TRY(check_rows(what, "v", v, v_stride, width, dtype));
    Q4_TRY(check_index(what, "slots", slots));
    DeviceInfo di;
    KvRowsArgs a = {*cache, const_cast<void*>(k), const_cast<void*>(v), slots, T, k_stride, v_stride, nullptr, log2_of(cache->page_size)};
    Q4_TRY(check_device_faults(what, &di, &a.fault));
    return finish(what, launch_kv4_write(a, dtype, (cudaStream_t)stream));
}

int kv4_read(void* k_out, void* v_out, const kv4_cache* cache, const int32_t* slots, int T, long long k_stride,
             long long v_stride, int dtype, q4_stream_t stream) {
    const char* what = "kv4_read";
    Q4_TRY(check_cache(what, cache));
    if (T <= 0 || T > (1 << 30)) return fail(Q4_EINVAL, "%s: T must be in 1..2^30 (got %d)", what, T);
    Q4_TRY(check_dtype(what, dtype));
    if (!k_out && !v_out) return fail(Q4_EINVAL, "%s: null k_out and v_out", what);
    const long long width = (long long)cache->num_kv_heads * cache->head_dim;
    if (k_out) Q4_TRY(check_rows(what, "k_out", k_out, k_stride, width, dtype));
    if (v_out) Q4_TRY(check_rows(what, "v_out", v_out, v_stride, width, dtype));
    Q4_TRY(check_index(what, "slots", slots));
    DeviceInfo di;
    KvRowsArgs a = {*cache, k_out, v_out, slots, T, k_stride, v_stride, nullptr, log2_of(cache->page_size)};
    Q4_TRY(check_device_faults(what, &di, &a.fault));
    return finish(what, launch_kv4_read(a, dtype, (cudaStream_t)stream));
}

static int check_attention_sizes(const char* what, int M, int Hq, int Hkv, int D, int dtype) {
    Q4_TRY(check_dtype(what, dtype));
    Q4_TRY(check_heads(what, Hkv, D));
    if (D != 64 && D != 128 && D != 256)
        return fail(Q4_EINVAL, "%s: the head size must be 64, 128 or 256 (got %d)", what, D);
    if (M < 1 || M > 16) return fail(Q4_EINVAL, "%s: M=%d outside 1..16 (refused, not clamped)", what, M);
    if (Hq <= 0 || Hq % Hkv != 0 || Hq > 65535)
        return fail(Q4_EINVAL, "%s: the query heads (%d) must be a multiple of the key heads (%d), up to 65535", what, Hq,
                    Hkv);
    return Q4_OK;
}

int kv4_attention_workspace(size_t* bytes, int M, int Hq, int Hkv, int D, int dtype) {
    const char* what = "kv4_attention_workspace";
    if (!bytes) return fail(Q4_EINVAL, "%s: null output pointer", what);
    Q4_TRY(check_attention_sizes(what, M, Hq, Hkv, D, dtype));
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    *bytes = kv4_attention_workspace_bytes(M, Hq / Hkv, Hkv, D, dtype, di.sm_count);
    return finish(what, cudaSuccess);
}

int kv4_attention(void* out, float* lse, const void* q, const kv4_cache* cache, const int32_t* block_table,
                  const int32_t* seq_lens, int B, int M, int Hq, int max_pages, long long q_stride, long long out_stride,
                  float scale, int window, int dtype, void* workspace, size_t workspace_bytes, q4_stream_t stream) {
    const char* what = "kv4_attention";
    Q4_TRY(check_cache(what, cache));
    Q4_TRY(check_attention_sizes(what, M, Hq, cache->num_kv_heads, cache->head_dim, dtype));
    if (B <= 0 || B > 1024) return fail(Q4_EINVAL, "%s: B must be in 1..1024 (got %d)", what, B);
    const long long width = (long long)Hq * cache->head_dim;
    Q4_TRY(check_rows(what, "q", q, q_stride, width, dtype));
    Q4_TRY(check_rows(what, "out", out, out_stride, width, dtype));
    if (lse && !aligned(lse, 4)) return fail(Q4_EALIGN, "%s: lse must be 4-byte aligned", what);
    Q4_TRY(check_index(what, "block_table", block_table));
    Q4_TRY(check_index(what, "seq_lens", seq_lens));
    if (max_pages <= 0 || (long long)max_pages * cache->page_size > (1LL << 30))
        return fail(Q4_EINVAL, "%s: max_pages must be >= 1 and hold up to 2^30 tokens (got %d)", what, max_pages);
    if (!(scale > 0.f) || !(scale <= 1e30f)) return fail(Q4_EINVAL, "%s: scale must be > 0 and at most 1e30", what);
    if (window < 0) return fail(Q4_EINVAL, "%s: window must be >= 0 (got %d)", what, window);
    if ((long long)window >= (long long)max_pages * cache->page_size) window = 0;  // it reaches past every sequence
    DeviceInfo di;
    KvAttnArgs a = {*cache, out, lse, q, block_table, seq_lens, B, M, Hq, max_pages, q_stride, out_stride, scale, window,
                    dtype, nullptr};
    Q4_TRY(check_device_faults(what, &di, &a.fault));
    const size_t need = kv4_attention_workspace_bytes(M, Hq / cache->num_kv_heads, cache->num_kv_heads, cache->head_dim, dtype, di.sm_count);
    if (need) {
        if (!workspace) return fail(Q4_EINVAL, "%s: null workspace", what);
        if (!aligned(workspace, 16)) return fail(Q4_EALIGN, "%s: workspace must be 16-byte aligned", what);
        if (workspace_bytes < need)
            return fail(Q4_EINVAL, "%s: the workspace holds %zu bytes, %zu are needed", what, workspace_bytes, need);
    }
    return finish(what, launch_kv4_attention(a, workspace, di, (cudaStream_t)stream));
}

int residual_norm(void* h_out, void* y_out, const void* x, const void* residual, const float* post_gamma, const void* gate,
                  const float* pre_gamma, float eps, float residual_scale, float branch_scale, int T, int K, int gate_width,
                  long long h_out_stride, long long y_out_stride, long long x_stride, long long residual_stride,
                  long long gate_stride, int dtype, q4_stream_t stream) {
    const char* what = "residual_norm";
    if (T <= 0) return fail(Q4_EINVAL, "%s: T must be >= 1 (got %d)", what, T);
    if (K <= 0 || K % 8 != 0 || K > 32768)
        return fail(Q4_EINVAL, "%s: K must be a multiple of 8 up to 32768 (got %d)", what, K);
    Q4_TRY(check_dtype(what, dtype));
    Q4_TRY(check_rows(what, "x", x, x_stride, K, dtype));
    Q4_TRY(check_rows(what, "h_out", h_out, h_out_stride, K, dtype));
    if ((y_out != nullptr) != (pre_gamma != nullptr))
        return fail(Q4_EINVAL, "%s: y_out and pre_gamma come together", what);
    if (y_out) Q4_TRY(check_rows(what, "y_out", y_out, y_out_stride, K, dtype));
    if (y_out == h_out) return fail(Q4_EINVAL, "%s: y_out and h_out are the same", what);
    if (residual) Q4_TRY(check_rows(what, "residual", residual, residual_stride, K, dtype));
    if (post_gamma) Q4_TRY(check_vec(what, "post_gamma", post_gamma));
    if (pre_gamma) Q4_TRY(check_vec(what, "pre_gamma", pre_gamma));
    if (gate) {
        if (gate_width != 1 && gate_width != K)
            return fail(Q4_EINVAL, "%s: gate_width must be K or 1 (got %d)", what, gate_width);
        if (gate_stride < 0 || (gate_stride > 0 && gate_stride < gate_width))
            return fail(Q4_EINVAL, "%s: token stride of gate is %lld, below its row of %d elements", what, gate_stride, gate_width);
        if (gate_width == K ? !aligned(gate, 16) || (gate_stride * (long long)dtype_bytes(dtype)) % 16 != 0
                            : !aligned(gate, dtype_bytes(dtype)))
            return fail(Q4_EALIGN, "%s: every row of gate must be 16-byte aligned", what);
    }
    Q4_TRY(check_eps(what, eps));
    if (!std::isfinite(residual_scale) || !std::isfinite(branch_scale))
        return fail(Q4_EINVAL, "%s: the scales must be finite", what);
    DeviceInfo di;
    Q4_TRY(check_device(what, &di));
    const ResidualNormArgs a = {h_out, y_out, x, residual, gate, post_gamma, pre_gamma, eps, residual_scale, branch_scale, T, K,
                                gate_width, h_out_stride, y_out_stride, x_stride, residual_stride, gate_stride, di.sm_count};
    return finish(what, launch_residual_norm(a, dtype, (cudaStream_t)stream));
}

// Sizes of a mixture of experts: `rows` and `cols` of a matrix, slots T * topk.
static int check_slots(const char* what, int T, int topk, int E) {
    if (E <= 0) return fail(Q4_EINVAL, "%s: E must be >= 1 (got %d)", what, E);
    if (T <= 0 || topk <= 0) return fail(Q4_EINVAL, "%s: T and topk must be >= 1", what);
    if (topk > E) return fail(Q4_EINVAL, "%s: topk=%d exceeds E=%d", what, topk, E);
    if ((long long)T * topk > 512) return fail(Q4_EINVAL, "%s: T*topk=%lld exceeds 512", what, (long long)T * topk);
    return Q4_OK;
}

static int check_down_sizes(const char* what, int T, int topk, int E, int N, int K) {
    Q4_TRY(check_slots(what, T, topk, E));
    if (N <= 0 || N % 8 != 0 || N > (1 << 20))
        return fail(Q4_EINVAL, "%s: N must be a multiple of 8 up to 2^20 (got %d)", what, N);
    if (K <= 0 || K % 32 != 0 || K > 65536)
        return fail(Q4_EINVAL, "%s: K must be a multiple of 32 up to 65536 (got %d)", what, K);
    if ((long long)E * N > 0x7fffffffLL) return fail(Q4_EINVAL, "%s: E*N exceeds 2^31-1 rows", what);
    return Q4_OK;
}

static int check_workspace(const char* what, const void* workspace, size_t bytes, size_t need) {
    if (!workspace) return fail(Q4_EINVAL, "%s: null workspace", what);
    if (!aligned(workspace, 16)) return fail(Q4_EALIGN, "%s: workspace must be 16-byte aligned", what);
    if (bytes < need) return fail(Q4_EINVAL, "%s: the workspace holds %zu bytes, %zu are needed", what, bytes, need);
    return Q4_OK;
}

int moe_q4_down_workspace(size_t* bytes, int T, int topk, int N, int K) {
    const char* what = "moe_q4_down_workspace";
    if (!bytes) return fail(Q4_EINVAL, "%s: null output pointer", what);
    Q4_TRY(check_down_sizes(what, T, topk, topk, N, K));
    *bytes = moe_down_workspace_bytes(T, topk, N, K);
    return finish(what, cudaSuccess);
}

int moe_q4_down_gemv(void* out, const uint8_t* qs, const uint16_t* d, const float* h, const int32_t* expert_ids,
                     const float* expert_weights, const void* residual, int T, int topk, int E, int N, int K,
                     long long out_stride, long long residual_stride, int dtype, int32_t* dev_status, void* workspace,
                     size_t workspace_bytes, q4_stream_t stream) {
    const char* what = "moe_q4_down_gemv";
    Q4_TRY(check_dtype(what, dtype));
    Q4_TRY(check_down_sizes(what, T, topk, E, N, K));
    Q4_TRY(check_rows(what, "out", out, out_stride, N, dtype));
    if (residual) Q4_TRY(check_rows(what, "residual", residual, residual_stride, N, dtype));
    Q4_TRY(check_q4_weights(what, qs, d, N, K));
    Q4_TRY(check_vec(what, "h", h));
    Q4_TRY(check_index(what, "expert_ids", expert_ids));
    if (!expert_weights) return fail(Q4_EINVAL, "%s: null expert_weights", what);
    if (!aligned(expert_weights, 4)) return fail(Q4_EALIGN, "%s: expert_weights must be 4-byte aligned", what);
    if (dev_status && !aligned(dev_status, 4)) return fail(Q4_EALIGN, "%s: dev_status must be 4-byte aligned", what);
    Q4_TRY(check_workspace(what, workspace, workspace_bytes, moe_down_workspace_bytes(T, topk, N, K)));
    DeviceInfo di;
    MoeDownArgs a = {out, qs, d, h, expert_ids, expert_weights, residual, T, topk, E, N, K, out_stride, residual_stride,
                     dev_status, nullptr};
    Q4_TRY(check_device_faults(what, &di, &a.fault));
    return finish(what, launch_moe_down(a, dtype, workspace, di, (cudaStream_t)stream));
}

static int check_layer_sizes(const char* what, int T, int topk, int E, int N, int K) {
    Q4_TRY(check_slots(what, T, topk, E));
    if (E > 4096) return fail(Q4_EINVAL, "%s: E must be in 1..4096 (got %d)", what, E);
    if (N <= 0 || N % 32 != 0 || N > 65536)
        return fail(Q4_EINVAL, "%s: N must be a multiple of 32 up to 65536 (got %d)", what, N);
    if (K <= 0 || K % 32 != 0 || K > 32768)
        return fail(Q4_EINVAL, "%s: K must be a multiple of 32 up to 32768 (got %d)", what, K);
    return Q4_OK;
}

int moe_q4_layer_workspace(size_t* bytes, int T, int topk, int E, int N, int K) {
    const char* what = "moe_q4_layer_workspace";
    if (!bytes) return fail(Q4_EINVAL, "%s: null output pointer", what);
    Q4_TRY(check_layer_sizes(what, T, topk, E, N, K));
    *bytes = moe_layer_workspace_bytes(T, topk, N, K);
    return finish(what, cudaSuccess);
}

int moe_q4_layer(void* out, const void* x, const moe_q4_weights* weights, const float* gamma, float eps, const void* residual,
                 int32_t* expert_ids, float* expert_weights, int T, int topk, int normalize, long long out_stride,
                 long long x_stride, long long residual_stride, int dtype, void* workspace, size_t workspace_bytes,
                 q4_stream_t stream) {
    const char* what = "moe_q4_layer";
    if (!weights) return fail(Q4_EINVAL, "%s: null weights", what);
    const moe_q4_weights& w = *weights;
    Q4_TRY(check_dtype(what, dtype));
    Q4_TRY(check_layer_sizes(what, T, topk, w.E, w.N, w.K));
    Q4_TRY(check_q4_weights(what, w.router_qs, w.router_d, w.E, w.K));
    Q4_TRY(check_q4_weights(what, w.gate_qs, w.gate_d, w.N, w.K));
    Q4_TRY(check_q4_weights(what, w.up_qs, w.up_d, w.N, w.K));
    Q4_TRY(check_q4_weights(what, w.down_qs, w.down_d, w.K, w.N));
    Q4_TRY(check_rows(what, "out", out, out_stride, w.K, dtype));
    Q4_TRY(check_rows(what, "x", x, x_stride, w.K, dtype));
    if (residual) Q4_TRY(check_rows(what, "residual", residual, residual_stride, w.K, dtype));
    if (gamma) Q4_TRY(check_vec(what, "gamma", gamma));
    Q4_TRY(check_eps(what, eps));
    if (!aligned(expert_ids, 4) || !aligned(expert_weights, 4))
        return fail(Q4_EALIGN, "%s: expert_ids and expert_weights must be 4-byte aligned", what);
    Q4_TRY(check_workspace(what, workspace, workspace_bytes, moe_layer_workspace_bytes(T, topk, w.N, w.K)));
    DeviceInfo di;
    MoeLayerArgs a = {w, out, x, residual, gamma, eps, T, topk, normalize != 0, out_stride, x_stride, residual_stride,
                      expert_ids, expert_weights, nullptr};
    Q4_TRY(check_device_faults(what, &di, &a.fault));
    return finish(what, launch_moe_layer(a, dtype, workspace, di, (cudaStream_t)stream));
}

const char* q4_last_error(void) { return g_last_error.c_str(); }

int q4_set_launch_overlap(int enable) {
    g_launch_overlap.store(enable ? 1 : 0, std::memory_order_relaxed);
    return Q4_OK;
}

int q4_get_launch_overlap(void) { return g_launch_overlap.load(std::memory_order_relaxed); }

int q4_device_faults(unsigned* faults) {
    const char* what = "q4_device_faults";
    if (!faults) return fail(Q4_EINVAL, "%s: null output pointer", what);
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(what, e);
    unsigned f = 0;
    if ((e = read_and_clear_faults(&f)) != cudaSuccess) return cuda_fail(what, e);
    *faults |= f;
    return finish(what, cudaSuccess);
}

int q4_set_wait_limit(long long cycles) {
    if (cycles < 0) return fail(Q4_EINVAL, "q4_set_wait_limit: the limit must be >= 0 (got %lld)", cycles);
    g_wait_limit.store(cycles, std::memory_order_relaxed);
    g_last_error.clear();
    return Q4_OK;
}

long long q4_get_wait_limit(void) { return g_wait_limit.load(std::memory_order_relaxed); }

}  // extern "C"
