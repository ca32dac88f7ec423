// qk_api.cu -- the extern "C" entry points of libqk (include/qk.h): argument
// validation on the host, then a launch on the caller's stream.  Nothing here
// allocates device memory; scratch comes from the caller's workspace.
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

#include "../../include/qk.h"
#include "qk_internal.h"

namespace {

thread_local std::string g_last_error;

// Kernel status word (bit 0: a bounded wait ran out).  One per device; its
// address is looked up once per device and passed to the kernels.
__device__ unsigned g_status_word;

constexpr int kMaxDevices = 64;
std::mutex g_mu;
unsigned* g_status_ptr[kMaxDevices] = {};
int g_sm_count[kMaxDevices] = {};

qk_status fail(qk_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
qk_status fail(qk_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

qk_status cuda_fail(cudaError_t e, const char* where) {
    return fail(QK_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool known_type(int t) { return t >= QK_Q4_K && t <= QK_Q3_K; }

size_t block_bytes(int t) {
    switch (t) {
    case QK_Q4_K: return 144;
    case QK_Q6_K: return 210;
    case QK_Q8_0: return 34;
    case QK_Q5_0: return 22;
    case QK_Q4_0: return 18;
    case QK_Q5_K: return 176;
    case QK_Q2_K: return 84;
    case QK_Q3_K: return 110;
    }
    return 0;
}

int block_elems(int t) {
    switch (t) {
    case QK_Q4_K: case QK_Q6_K: case QK_Q5_K: case QK_Q2_K: case QK_Q3_K: return 256;
    case QK_Q8_0: case QK_Q5_0: case QK_Q4_0: return 32;
    }
    return 0;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Per-device state: status-word address and SM count, set up on first use.
qk_status device_state(unsigned** status, int* sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(QK_ERR_ARG, "device %d out of range", dev);
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_status_ptr[dev]) {
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_status_word);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(status)");
        int n = 0;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
        g_sm_count[dev] = n;
        g_status_ptr[dev] = static_cast<unsigned*>(p);
    }
    if (status) *status = g_status_ptr[dev];
    if (sms) *sms = g_sm_count[dev];
    return QK_OK;
}

int sm_count_or_default() {
    int sms = 0;
    if (device_state(nullptr, &sms) != QK_OK || sms <= 0) return 148;
    return sms;
}

// Shared validation of (type, rows, cols, W).
qk_status check_matrix(int type, const void* W, int64_t rows, int64_t cols) {
    if (!known_type(type)) return fail(QK_ERR_TYPE, "unknown quant type %d", type);
    if (rows < 0 || cols < 0) return fail(QK_ERR_SHAPE, "negative shape rows=%lld cols=%lld", (long long)rows,
                                          (long long)cols);
    if (cols % block_elems(type) != 0)
        return fail(QK_ERR_SHAPE, "cols=%lld is not a multiple of %d", (long long)cols, block_elems(type));
    if (rows > 0 && cols > 0) {
        if (!W) return fail(QK_ERR_NULL, "W is NULL");
        if (!aligned(W, 16)) return fail(QK_ERR_ALIGN, "W is not 16-byte aligned");
    }
    return QK_OK;
}

bool kv_type(int t) { return t == QK_Q8_0 || t == QK_Q5_0 || t == QK_Q4_0; }

// log2 of a page size the paged cache takes, else -1.
int page_log2(int page) {
    for (int l = 4; l <= 8; ++l)
        if (page == 1 << l) return l;
    return -1;
}

// The most any count or stride of the paged calls may be (products of two of
// them, and of one with a row's bytes, stay inside 63 bits).
constexpr int64_t kCountMax = 0x7fffffff;
bool count_ok(int64_t n) { return n >= 0 && n <= kCountMax; }

// Shared validation of a paged pool's geometry and pointers.
qk_status check_pool(int type, int n_kv, int d, int page, int64_t n_pages, const void* K, const void* V) {
    if (!kv_type(type)) return fail(QK_ERR_TYPE, "KV cache type %d: Q8_0, Q5_0 or Q4_0 expected", type);
    if (n_kv < 1 || n_kv > 4096 || (d != 32 && d != 64 && d != 128 && d != 256))
        return fail(QK_ERR_SHAPE, "bad KV rows n_kv=%d d=%d", n_kv, d);
    if (page_log2(page) < 0) return fail(QK_ERR_SHAPE, "page=%d: 16, 32, 64, 128 or 256 expected", page);
    if (!count_ok(n_pages)) return fail(QK_ERR_SHAPE, "bad n_pages=%lld", (long long)n_pages);
    if (!K || !V) return fail(QK_ERR_NULL, "a KV pool is NULL");
    if (!aligned(K, 16) || !aligned(V, 16)) return fail(QK_ERR_ALIGN, "the KV pools must be 16-byte aligned");
    return QK_OK;
}

}  // namespace

namespace qk {
// Record `msg` as the calling thread's last error and return `st` (for entry
// points defined in other translation units).
qk_status set_error(qk_status st, const char* msg) { return fail(st, "%s", msg); }

// The argument checks of qk_gemv, in its order (no launch, no device call).
qk_status gemv_check_args(int type, const void* W, int64_t rows, int64_t cols, const float* x, int64_t M,
                          const float* y) {
    qk_status st = check_matrix(type, W, rows, cols);
    if (st != QK_OK) return st;
    if (M < 0) return fail(QK_ERR_SHAPE, "negative M=%lld", (long long)M);
    if (rows == 0 || M == 0) return QK_OK;
    if (!y) return fail(QK_ERR_NULL, "y is NULL");
    if (!aligned(y, 4)) return fail(QK_ERR_ALIGN, "y is not 4-byte aligned");
    if (cols == 0) return QK_OK;
    if (!x) return fail(QK_ERR_NULL, "x is NULL");
    if (!aligned(x, 16)) return fail(QK_ERR_ALIGN, "x is not 16-byte aligned");
    return QK_OK;
}
}  // namespace qk

extern "C" {

int qk_version(void) { return 1; }

size_t qk_block_bytes(int type) { return block_bytes(type); }

int qk_block_elems(int type) { return block_elems(type); }

size_t qk_row_bytes(int type, int64_t cols) {
    if (!known_type(type) || cols < 0 || cols % block_elems(type) != 0) return 0;
    return (size_t)(cols / block_elems(type)) * block_bytes(type);
}

const char* qk_last_error(void) { return g_last_error.c_str(); }

qk_status qk_dequant(int type, const void* W, int64_t rows, int64_t cols, void* out, int out_dtype, void* stream) {
    qk_status st = check_matrix(type, W, rows, cols);
    if (st != QK_OK) return st;
    if (out_dtype != QK_OUT_F32 && out_dtype != QK_OUT_BF16) return fail(QK_ERR_ARG, "bad out_dtype %d", out_dtype);
    if (rows == 0 || cols == 0) return QK_OK;
    if (!out) return fail(QK_ERR_NULL, "out is NULL");
    if (!aligned(out, 16)) return fail(QK_ERR_ALIGN, "out is not 16-byte aligned");
    cudaError_t e = qk::launch_dequant(type, static_cast<const uint8_t*>(W), rows, cols, out,
                                       out_dtype == QK_OUT_BF16, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_dequant launch");
    g_last_error.clear();
    return QK_OK;
}

qk_status qk_quantize(int type, const float* w, int64_t rows, int64_t cols, void* out, void* stream) {
    if (!known_type(type)) return fail(QK_ERR_TYPE, "unknown type %d", type);
    if (rows < 0 || cols < 0 || cols % block_elems(type) != 0)
        return fail(QK_ERR_SHAPE, "bad shape rows=%lld cols=%lld", (long long)rows, (long long)cols);
    if (rows == 0 || cols == 0) return QK_OK;
    if (rows > (int64_t(1) << 46) / cols)   // 2^46 weights: far beyond any device memory
        return fail(QK_ERR_SHAPE, "rows * cols too large (rows=%lld cols=%lld)", (long long)rows, (long long)cols);
    if (!w) return fail(QK_ERR_NULL, "w is NULL");
    if (!out) return fail(QK_ERR_NULL, "out is NULL");
    if (!aligned(w, 16)) return fail(QK_ERR_ALIGN, "w is not 16-byte aligned");
    if (!aligned(out, 4)) return fail(QK_ERR_ALIGN, "out is not 4-byte aligned");
    int sms = 0;
    const qk_status st = device_state(nullptr, &sms);
    if (st != QK_OK) return st;
    cudaError_t e = qk::launch_quantize(type, w, rows, cols, static_cast<uint8_t*>(out), sms,
                                        static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_quantize launch");
    g_last_error.clear();
    return QK_OK;
}

qk_status qk_quantize_imatrix(int type, const float* w, int64_t rows, int64_t cols, const float* imp, void* out,
                              void* stream) {
    if (!known_type(type)) return fail(QK_ERR_TYPE, "unknown type %d", type);
    if (rows < 0 || cols < 0 || cols % block_elems(type) != 0)
        return fail(QK_ERR_SHAPE, "bad shape rows=%lld cols=%lld", (long long)rows, (long long)cols);
    if (rows == 0 || cols == 0) return QK_OK;
    if (rows > (int64_t(1) << 46) / cols)
        return fail(QK_ERR_SHAPE, "rows * cols too large (rows=%lld cols=%lld)", (long long)rows, (long long)cols);
    if (!w) return fail(QK_ERR_NULL, "w is NULL");
    if (!imp) return fail(QK_ERR_NULL, "imp is NULL");
    if (!out) return fail(QK_ERR_NULL, "out is NULL");
    if (!aligned(w, 16)) return fail(QK_ERR_ALIGN, "w is not 16-byte aligned");
    if (!aligned(imp, 4) || !aligned(out, 4)) return fail(QK_ERR_ALIGN, "imp or out is not 4-byte aligned");
    cudaError_t e = qk::launch_quantize_imatrix(type, w, imp, rows, cols, static_cast<uint8_t*>(out),
                                               static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_quantize_imatrix launch");
    g_last_error.clear();
    return QK_OK;
}

size_t qk_attn_decode_workspace(int type, int64_t T, int n_heads, int n_kv, int d) {
    if ((type != QK_Q8_0 && type != QK_Q5_0 && type != QK_Q4_0) || T < 1 || !qk::attn_decode_shape_ok(n_heads, n_kv, d))
        return 0;
    return (size_t)qk::attn_decode_ws_bytes(T, n_heads, d);
}

qk_status qk_attn_decode(int type, const float* q, const void* K, const void* V, int64_t T, int n_heads, int n_kv, int d,
                         float scale, float* out, void* ws, size_t ws_bytes, void* stream) {
    if (type != QK_Q8_0 && type != QK_Q5_0 && type != QK_Q4_0)
        return fail(QK_ERR_TYPE, "KV cache type %d: Q8_0, Q5_0 or Q4_0 expected", type);
    if (T < 1 || T > (int64_t)65535 * 256 || !qk::attn_decode_shape_ok(n_heads, n_kv, d))
        return fail(QK_ERR_SHAPE, "bad attention shape T=%lld n_heads=%d n_kv=%d d=%d", (long long)T, n_heads, n_kv, d);
    if (!q || !K || !V || !out || !ws) return fail(QK_ERR_NULL, "NULL pointer argument");
    if (!aligned(q, 4) || !aligned(out, 4) || !aligned(ws, 4) || !aligned(K, 16) || !aligned(V, 16))
        return fail(QK_ERR_ALIGN, "q, out and ws must be 4-byte aligned, K and V 16-byte aligned");
    const int64_t need = qk::attn_decode_ws_bytes(T, n_heads, d);
    if (ws_bytes < (size_t)need) return fail(QK_ERR_WORKSPACE, "workspace %zu bytes < %lld needed", ws_bytes, (long long)need);
    unsigned* status = nullptr;
    int sms = 0;
    const qk_status st = device_state(&status, &sms);
    if (st != QK_OK) return st;
    cudaError_t e = qk::launch_attn_decode(type, q, static_cast<const uint8_t*>(K), static_cast<const uint8_t*>(V), T,
                                           n_heads, n_kv, d, scale, out, static_cast<float*>(ws), status, sms,
                                           static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_attn_decode launch");
    g_last_error.clear();
    return QK_OK;
}

size_t qk_gemv_workspace(int type, int64_t rows, int64_t cols, int64_t M) {
    if (!known_type(type) || rows <= 0 || cols <= 0 || M <= 0 || cols % block_elems(type) != 0) return 0;
    return (size_t)qk::plan_gemv(type, rows, cols, M, sm_count_or_default()).ws_bytes;
}

qk_status qk_gemv(int type, const void* W, int64_t rows, int64_t cols, const float* x, int64_t M, float* y,
                  void* ws, size_t ws_bytes, void* stream) {
    qk_status st = qk::gemv_check_args(type, W, rows, cols, x, M, y);
    if (st != QK_OK) return st;
    if (rows == 0 || M == 0) return QK_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cols == 0) {
        cudaError_t e = cudaMemsetAsync(y, 0, (size_t)(M * rows) * sizeof(float), s);
        if (e != cudaSuccess) return cuda_fail(e, "qk_gemv zero fill");
        return QK_OK;
    }
    unsigned* status = nullptr;
    int sms = 0;
    st = device_state(&status, &sms);
    if (st != QK_OK) return st;
    (void)ws;   // no shape needs one
    (void)ws_bytes;
    const qk::GemvPlan pl = qk::plan_gemv(type, rows, cols, M, sms);
    if (!pl.ok) return fail(QK_ERR_SHAPE, "rows=%lld cols=%lld: no GEMV launch fits", (long long)rows, (long long)cols);
    cudaError_t e = qk::launch_gemv(type, pl, static_cast<const uint8_t*>(W), rows, cols, x, M, y, status, s);
    if (e != cudaSuccess) return cuda_fail(e, "qk_gemv launch");
    g_last_error.clear();
    return QK_OK;
}

qk_status qk_gemv_batch(int type, int n_mat, const void* const* W, const int64_t* rows, int64_t cols,
                        const float* x, float* const* y, void* stream) {
    if (!known_type(type)) return fail(QK_ERR_TYPE, "unknown quant type %d", type);
    if (n_mat < 1 || n_mat > QK_GEMV_BATCH_MAX)
        return fail(QK_ERR_ARG, "n_mat=%d outside 1..%d", n_mat, QK_GEMV_BATCH_MAX);
    if (!W || !rows || !y) return fail(QK_ERR_NULL, "W, rows or y array is NULL");
    int64_t total = 0;
    for (int i = 0; i < n_mat; ++i) {
        qk_status st = check_matrix(type, W[i], rows[i], cols);
        if (st != QK_OK) return st;
        if (rows[i] > 0) {
            if (!y[i]) return fail(QK_ERR_NULL, "y[%d] is NULL", i);
            if (!aligned(y[i], 4)) return fail(QK_ERR_ALIGN, "y[%d] is not 4-byte aligned", i);
        }
        total += rows[i];
    }
    if (total == 0) return QK_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cols == 0) {
        for (int i = 0; i < n_mat; ++i) {
            if (rows[i] == 0) continue;
            cudaError_t e = cudaMemsetAsync(y[i], 0, (size_t)rows[i] * sizeof(float), s);
            if (e != cudaSuccess) return cuda_fail(e, "qk_gemv_batch zero fill");
        }
        return QK_OK;
    }
    if (!x) return fail(QK_ERR_NULL, "x is NULL");
    if (!aligned(x, 16)) return fail(QK_ERR_ALIGN, "x is not 16-byte aligned");
    int sms = 0;
    unsigned* status = nullptr;
    qk_status st = device_state(&status, &sms);
    if (st != QK_OK) return st;
    cudaError_t e;
    if (!qk::hgemv_ok(type, n_mat, rows, cols, sms))
        return fail(QK_ERR_SHAPE, "cols=%lld: no batched GEMV launch fits", (long long)cols);
    e = qk::launch_hgemv(type, n_mat, reinterpret_cast<const uint8_t* const*>(W), rows, cols, x, y, sms, status, s);
    if (e != cudaSuccess) return cuda_fail(e, "qk_gemv_batch launch");
    g_last_error.clear();
    return QK_OK;
}

qk_status qk_gemv_swiglu(int type, const void* Wg, const void* Wu, int64_t rows, int64_t cols, const float* x,
                         float* h, void* stream) {
    qk_status st = check_matrix(type, Wg, rows, cols);
    if (st != QK_OK) return st;
    st = check_matrix(type, Wu, rows, cols);
    if (st != QK_OK) return st;
    if (rows == 0) return QK_OK;
    if (!h) return fail(QK_ERR_NULL, "h is NULL");
    if (!aligned(h, 4)) return fail(QK_ERR_ALIGN, "h is not 4-byte aligned");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cols == 0) {   // g = u = 0, SiLU(0) * 0 = 0
        cudaError_t e = cudaMemsetAsync(h, 0, (size_t)rows * sizeof(float), s);
        if (e != cudaSuccess) return cuda_fail(e, "qk_gemv_swiglu zero fill");
        return QK_OK;
    }
    if (!x) return fail(QK_ERR_NULL, "x is NULL");
    if (!aligned(x, 16)) return fail(QK_ERR_ALIGN, "x is not 16-byte aligned");
    int sms = 0;
    unsigned* status = nullptr;
    st = device_state(&status, &sms);
    if (st != QK_OK) return st;
    if (!qk::hgemv_ok(type, 1, &rows, cols, sms))
        return fail(QK_ERR_SHAPE, "rows=%lld cols=%lld: no SwiGLU launch fits", (long long)rows, (long long)cols);
    const cudaError_t e = qk::launch_hgemv_swiglu(type, static_cast<const uint8_t*>(Wg), static_cast<const uint8_t*>(Wu),
                                                  rows, cols, x, h, sms, status, s);
    if (e != cudaSuccess) return cuda_fail(e, "qk_gemv_swiglu launch");
    g_last_error.clear();
    return QK_OK;
}

size_t qk_gemm_workspace(int type, int64_t rows, int64_t cols, int64_t M) {
    if (!known_type(type) || rows <= 0 || cols <= 0 || M <= 0 || cols % block_elems(type) != 0) return 0;
    return (size_t)qk::plan_gemm(type, rows, cols, M, sm_count_or_default()).ws_bytes;
}

qk_status qk_gemm(int type, const void* W, int64_t rows, int64_t cols, const void* X_bf16, int64_t M, float* Y,
                  void* ws, size_t ws_bytes, void* stream) {
    qk_status st = check_matrix(type, W, rows, cols);
    if (st != QK_OK) return st;
    if (M < 0) return fail(QK_ERR_SHAPE, "negative M=%lld", (long long)M);
    if (rows == 0 || M == 0) return QK_OK;
    if (!Y) return fail(QK_ERR_NULL, "Y is NULL");
    if (!aligned(Y, 4)) return fail(QK_ERR_ALIGN, "Y is not 4-byte aligned");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cols == 0) {
        cudaError_t e = cudaMemsetAsync(Y, 0, (size_t)(M * rows) * sizeof(float), s);
        if (e != cudaSuccess) return cuda_fail(e, "qk_gemm zero fill");
        return QK_OK;
    }
    if (!X_bf16) return fail(QK_ERR_NULL, "X is NULL");
    if (!aligned(X_bf16, 16)) return fail(QK_ERR_ALIGN, "X is not 16-byte aligned");
    if (rows > (int64_t)1 << 31 || M > (int64_t)1 << 31 || cols > (int64_t)1 << 31)
        return fail(QK_ERR_SHAPE, "qk_gemm: dimensions must be below 2^31");
    if ((rows + 127) / 128 > 65535)
        return fail(QK_ERR_SHAPE, "qk_gemm: rows=%lld above 65535 tiles of 128", (long long)rows);
    unsigned* status = nullptr;
    int sms = 0;
    st = device_state(&status, &sms);
    if (st != QK_OK) return st;
    const qk::GemmPlan pl = qk::plan_gemm(type, rows, cols, M, sms);
    if (pl.ws_bytes > 0) {
        if (ws_bytes < (size_t)pl.ws_bytes)
            return fail(QK_ERR_WORKSPACE, "workspace %zu bytes < %lld needed", ws_bytes, (long long)pl.ws_bytes);
        if (!ws) return fail(QK_ERR_NULL, "workspace is NULL");
        if (!aligned(ws, 16)) return fail(QK_ERR_ALIGN, "workspace is not 16-byte aligned");
    }
    cudaError_t e = qk::launch_gemm(type, pl, static_cast<const uint8_t*>(W), rows, cols, X_bf16, M, Y,
                                    static_cast<float*>(ws), status, s);
    if (e != cudaSuccess) return cuda_fail(e, "qk_gemm launch");
    g_last_error.clear();
    return QK_OK;
}

qk_status qk_unpack(int type, const void* W, int64_t nblocks, int16_t* codes, int16_t* sc, uint8_t* mins, float* d,
                    float* dmin, void* stream) {
    if (!known_type(type)) return fail(QK_ERR_TYPE, "unknown quant type %d", type);
    if (nblocks < 0) return fail(QK_ERR_SHAPE, "negative nblocks");
    if (nblocks == 0) return QK_OK;
    if (!W) return fail(QK_ERR_NULL, "W is NULL");
    if (!aligned(W, 16)) return fail(QK_ERR_ALIGN, "W is not 16-byte aligned");
    cudaError_t e = qk::launch_unpack(type, static_cast<const uint8_t*>(W), nblocks, codes, sc, mins, d, dmin,
                                      static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_unpack launch");
    return QK_OK;
}

qk_status qk_test_stalled_wait(uint32_t limit_us, void* stream) {
    if (limit_us < 1 || limit_us > 10000000u) return fail(QK_ERR_ARG, "limit_us=%u outside 1..10000000", limit_us);
    unsigned* status = nullptr;
    qk_status st = device_state(&status, nullptr);
    if (st != QK_OK) return st;
    cudaError_t e = qk::launch_stalled_wait(status, (uint64_t)limit_us * 1000u, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_test_stalled_wait launch");
    g_last_error.clear();
    return QK_OK;
}

// --- the paged KV cache, tree attention over it, logits ---

size_t qk_kv_page_bytes(int type, int n_kv, int d, int page) {
    if (!kv_type(type) || n_kv < 1 || n_kv > 4096 || (d != 32 && d != 64 && d != 128 && d != 256) || page_log2(page) < 0)
        return 0;
    return (size_t)n_kv * page * (d / 32) * block_bytes(type);
}

qk_status qk_kv_plan(const int32_t* have, const int32_t* start, const int32_t* want, int64_t n_req, int page,
                     int32_t* table, int64_t table_stride, int32_t* free_pages, int64_t free_cap, const int32_t* n_free,
                     int32_t* n_free_out, int32_t* granted, int32_t* cu, int64_t* slots, int32_t* pos, int32_t* req,
                     int64_t cap, void* stream) {
    if (n_req < 0 || n_req > QK_PLAN_MAX_REQ)
        return fail(QK_ERR_SHAPE, "n_req=%lld outside 0..%d", (long long)n_req, QK_PLAN_MAX_REQ);
    if (page_log2(page) < 0) return fail(QK_ERR_SHAPE, "page=%d: 16, 32, 64, 128 or 256 expected", page);
    if (!count_ok(table_stride) || !count_ok(free_cap) || !count_ok(cap))
        return fail(QK_ERR_SHAPE, "bad table_stride=%lld, free_cap=%lld or cap=%lld", (long long)table_stride,
                    (long long)free_cap, (long long)cap);
    if (!n_free || !n_free_out || !cu || (n_req > 0 && (!have || !start || !want || !granted)) ||
        (n_req > 0 && table_stride > 0 && !table) || (free_cap > 0 && !free_pages) || (cap > 0 && !slots))
        return fail(QK_ERR_NULL, "NULL pointer argument");
    for (const void* p : {(const void*)have, (const void*)start, (const void*)want, (const void*)table,
                          (const void*)free_pages, (const void*)n_free, (const void*)n_free_out, (const void*)granted,
                          (const void*)cu, (const void*)pos, (const void*)req})
        if (!aligned(p, 4)) return fail(QK_ERR_ALIGN, "the int32 arrays must be 4-byte aligned");
    if (!aligned(slots, 8)) return fail(QK_ERR_ALIGN, "slots must be 8-byte aligned");
    if (n_free == n_free_out) return fail(QK_ERR_ARG, "n_free_out must not be n_free");
    int sms = 0;
    const qk_status st = device_state(nullptr, &sms);
    if (st != QK_OK) return st;
    cudaError_t e = qk::launch_kv_plan(have, start, want, (int)n_req, page_log2(page), table, table_stride, free_pages,
                                       free_cap, n_free, n_free_out, granted, cu, slots, pos, req, cap, sms,
                                       static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_kv_plan launch");
    g_last_error.clear();
    return QK_OK;
}

qk_status qk_kv_append(int type, const void* k, const void* v, int dtype, int64_t n_tok, int64_t k_stride, int64_t v_stride,
                       int n_kv, int d, const int64_t* slots, void* K, void* V, int64_t n_pages, int page, void* stream) {
    qk_status st = check_pool(type, n_kv, d, page, n_pages, K, V);
    if (st != QK_OK) return st;
    if (dtype != QK_OUT_F32 && dtype != QK_OUT_BF16) return fail(QK_ERR_ARG, "bad dtype %d", dtype);
    const int64_t row = (int64_t)n_kv * d;
    // the launch's grid: 64 blocks of 32 elements a CTA
    if (n_tok < 0 || n_tok > (int64_t(1) << 31) * 32 / row)
        return fail(QK_ERR_SHAPE, "bad n_tok=%lld", (long long)n_tok);
    if (n_tok == 0) return QK_OK;
    if (k_stride < row || v_stride < row || !count_ok(k_stride) || !count_ok(v_stride))
        return fail(QK_ERR_SHAPE, "bad strides k_stride=%lld v_stride=%lld", (long long)k_stride, (long long)v_stride);
    if (!k || !v || !slots) return fail(QK_ERR_NULL, "k, v or slots is NULL");
    const size_t es = dtype == QK_OUT_BF16 ? 2 : 4;
    if (!aligned(k, es) || !aligned(v, es) || !aligned(slots, 8))
        return fail(QK_ERR_ALIGN, "k and v must be aligned to their element, slots to 8 bytes");
    unsigned* status = nullptr;
    st = device_state(&status, nullptr);
    if (st != QK_OK) return st;
    cudaError_t e = qk::launch_kv_append(type, k, v, dtype == QK_OUT_BF16, n_tok, k_stride, v_stride, n_kv, d, slots,
                                         static_cast<uint8_t*>(K), static_cast<uint8_t*>(V), n_pages, page_log2(page),
                                         (int)qk_row_bytes(type, d), status, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_kv_append launch");
    g_last_error.clear();
    return QK_OK;
}

qk_status qk_kv_compact(int type, void* K, void* V, int64_t n_pages, int page, int n_kv, int d, const int32_t* table,
                        int64_t table_stride, const int32_t* base, const int32_t* path, int64_t path_stride,
                        const int32_t* n_path, int64_t n_req, void* stream) {
    qk_status st = check_pool(type, n_kv, d, page, n_pages, K, V);
    if (st != QK_OK) return st;
    if (!count_ok(n_req) || !count_ok(table_stride) || !count_ok(path_stride))
        return fail(QK_ERR_SHAPE, "bad n_req=%lld, table_stride=%lld or path_stride=%lld", (long long)n_req,
                    (long long)table_stride, (long long)path_stride);
    if (n_req == 0 || path_stride == 0) return QK_OK;
    if (!table || !base || !path || !n_path) return fail(QK_ERR_NULL, "NULL pointer argument");
    if (!aligned(table, 4) || !aligned(base, 4) || !aligned(path, 4) || !aligned(n_path, 4))
        return fail(QK_ERR_ALIGN, "the int32 arrays must be 4-byte aligned");
    unsigned* status = nullptr;
    st = device_state(&status, nullptr);
    if (st != QK_OK) return st;
    cudaError_t e = qk::launch_kv_compact(static_cast<uint8_t*>(K), static_cast<uint8_t*>(V), n_pages, page_log2(page),
                                          n_kv, (int)qk_row_bytes(type, d), table, table_stride, base, path, path_stride,
                                          n_path, n_req, status, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_kv_compact launch");
    g_last_error.clear();
    return QK_OK;
}

static bool attn_tree_shape_ok(int64_t n_req, int max_q, int64_t max_pos, int n_heads, int n_kv, int d) {
    return n_req >= 0 && n_req <= 65535 && max_q >= 1 && max_q <= QK_TREE_MAX && max_pos >= 0 &&
           max_pos <= kCountMax * 256 && n_kv >= 1 && n_kv <= 4096 && n_heads >= n_kv && n_heads % n_kv == 0 &&
           n_heads / n_kv <= 64 && (d == 32 || d == 64 || d == 128 || d == 256) &&
           qk::attn_tree_max_tiles(n_req, max_q, max_pos, n_heads, n_kv, d) < 2147000000.0;   // counted in 32 bits
}

size_t qk_attn_tree_workspace(int type, int64_t n_req, int max_q, int64_t max_pos, int n_heads, int n_kv, int d) {
    if (!kv_type(type) || !attn_tree_shape_ok(n_req, max_q, max_pos, n_heads, n_kv, d)) return 0;
    return (size_t)qk::attn_tree_ws_bytes(n_req, max_q, max_pos, n_heads, n_kv, d, sm_count_or_default());
}

static qk_status attn_tree(uint32_t looks, uint32_t hold, int type, const void* q, int64_t n_tok, int64_t q_stride,
                           const void* K, const void* V, int64_t n_pages, int page, const int32_t* table,
                           int64_t table_stride, const int32_t* ctx, const int32_t* cu, const uint64_t* mask, int64_t n_req,
                           int max_q, int n_heads, int n_kv, int d, float scale, void* out, int64_t out_stride, void* ws,
                           size_t ws_bytes, void* stream) {
    qk_status st = check_pool(type, n_kv, d, page, n_pages, K, V);
    if (st != QK_OK) return st;
    if (!count_ok(table_stride) || !count_ok(n_tok) ||
        !attn_tree_shape_ok(n_req, max_q, table_stride * page, n_heads, n_kv, d))
        return fail(QK_ERR_SHAPE, "bad attention shape n_req=%lld n_tok=%lld max_q=%d table_stride=%lld n_heads=%d n_kv=%d d=%d",
                    (long long)n_req, (long long)n_tok, max_q, (long long)table_stride, n_heads, n_kv, d);
    if (n_tok == 0 || n_req == 0) return QK_OK;
    const int64_t row = (int64_t)n_heads * d;
    if (q_stride < row || out_stride < row || !count_ok(q_stride) || !count_ok(out_stride))
        return fail(QK_ERR_SHAPE, "bad strides q_stride=%lld out_stride=%lld", (long long)q_stride, (long long)out_stride);
    if (!q || !out || !ctx || !cu || (table_stride > 0 && !table) || !ws) return fail(QK_ERR_NULL, "NULL pointer argument");
    if (!aligned(q, 16) || q_stride % 8 != 0)
        return fail(QK_ERR_ALIGN, "q must be 16-byte aligned and q_stride a multiple of 8");
    if (!aligned(out, 2) || !aligned(ws, 16) || !aligned(table, 4) || !aligned(ctx, 4) || !aligned(cu, 4) || !aligned(mask, 8))
        return fail(QK_ERR_ALIGN, "out must be 2-byte aligned, ws 16, the int32 arrays 4 and mask 8");
    const size_t need = qk_attn_tree_workspace(type, n_req, max_q, table_stride * page, n_heads, n_kv, d);
    if (ws_bytes < need) return fail(QK_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
    unsigned* status = nullptr;
    int sms = 0;
    st = device_state(&status, &sms);
    if (st != QK_OK) return st;
    cudaError_t e = qk::launch_attn_tree(type, q, n_tok, q_stride, static_cast<const uint8_t*>(K),
                                         static_cast<const uint8_t*>(V), n_pages, page_log2(page),
                                         (int)qk_row_bytes(type, d), table, table_stride, ctx, cu, mask, n_req, max_q,
                                         n_heads, n_kv, d, scale, out, out_stride, ws, status, looks, hold, sms,
                                         static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_attn_tree launch");
    g_last_error.clear();
    return QK_OK;
}

qk_status qk_attn_tree(int type, const void* q, int64_t n_tok, int64_t q_stride, const void* K, const void* V,
                       int64_t n_pages, int page, const int32_t* table, int64_t table_stride, const int32_t* ctx,
                       const int32_t* cu, const uint64_t* mask, int64_t n_req, int max_q, int n_heads, int n_kv, int d,
                       float scale, void* out, int64_t out_stride, void* ws, size_t ws_bytes, void* stream) {
    return attn_tree(qk::kTreeLooks, ~0u, type, q, n_tok, q_stride, K, V, n_pages, page, table, table_stride, ctx, cu,
                     mask, n_req, max_q, n_heads, n_kv, d, scale, out, out_stride, ws, ws_bytes, stream);
}

qk_status qk_test_attn_tree_stalled(uint32_t limit_us, uint32_t tile, int type, const void* q, int64_t n_tok,
                                    int64_t q_stride, const void* K, const void* V, int64_t n_pages, int page,
                                    const int32_t* table, int64_t table_stride, const int32_t* ctx, const int32_t* cu,
                                    const uint64_t* mask, int64_t n_req, int max_q, int n_heads, int n_kv, int d, float scale,
                                    void* out, int64_t out_stride, void* ws, size_t ws_bytes, void* stream) {
    if (limit_us < 1 || limit_us > 2000000) return fail(QK_ERR_ARG, "limit_us=%u outside 1..2000000", limit_us);
    return attn_tree((limit_us * 1000u + qk::kTreeLookNs - 1) / qk::kTreeLookNs, tile, type, q, n_tok, q_stride, K, V, n_pages, page, table, table_stride, ctx, cu, mask,
                     n_req, max_q, n_heads, n_kv, d, scale, out, out_stride, ws, ws_bytes, stream);
}

qk_status qk_logits_process(const void* logits, int dtype, int64_t n_rows, int64_t vocab, int64_t row_stride,
                            const int32_t* cu, int64_t n_req, const int32_t* hist, int64_t hist_stride,
                            const int32_t* hist_len, const float* rep, const float* pres, const float* freq,
                            const int32_t* draft, const uint64_t* mask, const int32_t* bias_tok, const float* bias_val,
                            int64_t bias_stride, const int32_t* bias_len, const uint32_t* grammar, int64_t grammar_stride,
                            void* out, int64_t out_stride, void* stream) {
    if (dtype != QK_OUT_F32 && dtype != QK_OUT_BF16) return fail(QK_ERR_ARG, "bad dtype %d", dtype);
    if (!count_ok(n_rows) || !count_ok(vocab) || !count_ok(n_req))
        return fail(QK_ERR_SHAPE, "bad n_rows=%lld, vocab=%lld or n_req=%lld", (long long)n_rows, (long long)vocab,
                    (long long)n_req);
    if (n_rows == 0 || vocab == 0) return QK_OK;
    if (row_stride < vocab || out_stride < vocab || !count_ok(row_stride) || !count_ok(out_stride))
        return fail(QK_ERR_SHAPE, "bad strides row_stride=%lld out_stride=%lld", (long long)row_stride, (long long)out_stride);
    if (hist_stride < 0 || hist_stride >= (1 << 20) - 64)
        return fail(QK_ERR_SHAPE, "hist_stride=%lld outside 0..2^20-65", (long long)hist_stride);
    if (bias_tok && (bias_stride < 0 || bias_stride > 4095))
        return fail(QK_ERR_SHAPE, "bias_stride=%lld outside 0..4095", (long long)bias_stride);
    if (grammar && (grammar_stride < (vocab + 31) / 32 || !count_ok(grammar_stride)))
        return fail(QK_ERR_SHAPE, "grammar_stride=%lld below vocab / 32", (long long)grammar_stride);
    if (!logits || !out || !cu || (n_req > 0 && (!hist_len || !rep || !pres || !freq || (hist_stride > 0 && !hist))) ||
        (bias_tok && (!bias_val || !bias_len)))
        return fail(QK_ERR_NULL, "NULL pointer argument");
    const size_t es = dtype == QK_OUT_BF16 ? 2 : 4;
    if (!aligned(logits, es) || !aligned(out, es)) return fail(QK_ERR_ALIGN, "logits and out must be aligned to their element");
    for (const void* p : {(const void*)cu, (const void*)hist, (const void*)hist_len, (const void*)rep, (const void*)pres,
                          (const void*)freq, (const void*)draft, (const void*)bias_tok, (const void*)bias_val,
                          (const void*)bias_len, (const void*)grammar})
        if (!aligned(p, 4)) return fail(QK_ERR_ALIGN, "the lists must be 4-byte aligned");
    if (!aligned(mask, 8)) return fail(QK_ERR_ALIGN, "mask must be 8-byte aligned");
    if (out == logits && out_stride != row_stride) return fail(QK_ERR_ARG, "in place needs out_stride == row_stride");
    unsigned* status = nullptr;
    int sms = 0;
    const qk_status st = device_state(&status, &sms);
    if (st != QK_OK) return st;
    const qk::LogitsArgs a{logits, dtype == QK_OUT_BF16, n_rows, vocab, row_stride, cu, n_req, hist, hist_stride, hist_len,
                           rep, pres, freq, draft, mask, bias_tok, bias_val, bias_stride, bias_len, grammar,
                           grammar_stride, out, out_stride, status};
    cudaError_t e = qk::launch_logits_process(a, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_logits_process launch");
    g_last_error.clear();
    return QK_OK;
}

qk_status qk_device_status(void* stream) {
    unsigned* status = nullptr;
    qk_status st = device_state(&status, nullptr);
    if (st != QK_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned v = 0;
    cudaError_t e = cudaMemcpyAsync(&v, status, sizeof v, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(status, 0, sizeof v, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "qk_device_status");
    if (v & 1u) return fail(QK_ERR_TIMEOUT, "a bounded wait inside a kernel ran out (status 0x%x)", v);
    if (v & 2u) return fail(QK_ERR_ARG, "a page id or slot outside its KV pool (status 0x%x)", v);
    if (v & 4u) return fail(QK_ERR_ARG, "a request's history and drafted tokens come to 2^20 or more (status 0x%x)", v);
    return QK_OK;
}

}  // extern "C"
