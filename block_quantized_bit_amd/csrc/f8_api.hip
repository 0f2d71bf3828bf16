// C entry points of the e4m3 product (f8.h): host-side validation, then launches.
#include "f8.h"
#include "kernels_wide.h"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
inline int up128(int v) { return (v + 127) / 128 * 128; }
int hip_status(hipError_t e) { return e == hipSuccess ? Q4_OK : Q4_ERR_HIP; }

constexpr int MOST = 1 << 22;             // each of M, N, K: rows of a tile stay within 32-bit offsets
constexpr long long MOST_CODES = 1LL << 34;  // codes of one operand: the quantizer's grid

bool size_ok(int a, int b) { return a > 0 && b > 0 && a <= MOST && b <= MOST && (long long)up128(a) * up128(b) <= MOST_CODES; }
// Outputs of one product: the tiles' grid stays below 2^32 threads.
bool product_ok(int M, int N) { return (long long)M * N <= (1LL << 37); }
bool type_ok(int dt) { return dt == Q4_DT_F32 || dt == Q4_DT_BF16; }
uintptr_t size_of(int dt) { return dt == Q4_DT_BF16 ? 2 : 4; }

size_t codes_bytes(int rows, int cols) { return align256((size_t)rows * up128(cols)); }
size_t scales_bytes(int rows, int cols) { return align256((size_t)rows * (up128(cols) / 128) * 4); }

int check_x(int M, int K, int dt, const void* x, long long stride) {
    if (!type_ok(dt)) return Q4_ERR_FORMAT;
    if (!size_ok(M, K) || stride < K || stride > (1LL << 40)) return Q4_ERR_DIM;
    if (!aligned(x, size_of(dt))) return Q4_ERR_ALIGN;
    return Q4_OK;
}

}  // namespace

extern "C" {

int f8_quantize_rows(int M, int K, int xdtype, const void* x, long long x_stride, uint8_t* xq, float* xs,
                     void* stream) {
    if (!x || !xq || !xs) return Q4_ERR_NULL;
    const int st = check_x(M, K, xdtype, x, x_stride);
    if (st) return st;
    if (!aligned(xq, 16) || !aligned(xs, 4)) return Q4_ERR_ALIGN;
    return hip_status(q4::launch_f8_quantize_rows(M, K, xdtype == Q4_DT_BF16, x, x_stride, xq, xs,
                                                  static_cast<hipStream_t>(stream)));
}

int f8_quantize_cols(int M, int K, int xdtype, const void* x, long long x_stride, uint8_t* xt, float* xts,
                     void* stream) {
    if (!x || !xt || !xts) return Q4_ERR_NULL;
    const int st = check_x(M, K, xdtype, x, x_stride);
    if (st) return st;
    if (!aligned(xt, 16) || !aligned(xts, 4)) return Q4_ERR_ALIGN;
    return hip_status(q4::launch_f8_quantize_cols(M, K, xdtype == Q4_DT_BF16, x, x_stride, xt, xts,
                                                  static_cast<hipStream_t>(stream)));
}

int f8_quantize_weights(int N, int K, int wdtype, const void* w, uint8_t* wq, float* ws, void* stream) {
    if (!w || !wq || !ws) return Q4_ERR_NULL;
    const int st = check_x(N, K, wdtype, w, K);
    if (st) return st;
    if (!aligned(wq, 16) || !aligned(ws, 4)) return Q4_ERR_ALIGN;
    return hip_status(q4::launch_f8_quantize_weights(N, K, wdtype == Q4_DT_BF16, w, wq, ws,
                                                     static_cast<hipStream_t>(stream)));
}

int f8_transpose_weights(int N, int K, const uint8_t* wq, const float* ws, uint8_t* wqt, float* wst, void* stream) {
    if (!wq || !ws || !wqt || !wst) return Q4_ERR_NULL;
    if (!size_ok(N, K)) return Q4_ERR_DIM;
    if (!aligned(wq, 16) || !aligned(wqt, 16) || !aligned(ws, 4) || !aligned(wst, 4)) return Q4_ERR_ALIGN;
    return hip_status(q4::launch_f8_transpose(N, K, wq, ws, wqt, wst, static_cast<hipStream_t>(stream)));
}

int f8_gemm(int M, int Kp, int N, int ydtype, const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
            void* y, void* stream) {
    if (!xq || !xs || !wq || !ws || !y) return Q4_ERR_NULL;
    if (!type_ok(ydtype)) return Q4_ERR_FORMAT;
    if (!size_ok(M, Kp) || !size_ok(N, Kp) || !product_ok(M, N)) return Q4_ERR_DIM;
    if (Kp % 128 != 0) return Q4_ERR_BLOCK;
    if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(y, 16) || !aligned(xs, 4) || !aligned(ws, 4))
        return Q4_ERR_ALIGN;
    return hip_status(q4::launch_f8_gemm(M, N, Kp / 128, ydtype == Q4_DT_BF16, xq, xs, wq, ws, y,
                                         static_cast<hipStream_t>(stream)));
}

size_t f8_linear_work_bytes(int M, int K) {
    if (!size_ok(M, K)) return 0;
    return codes_bytes(M, K) + scales_bytes(M, K);
}

int f8_linear(int M, int K, int N, int xdtype, const void* x, long long x_stride, const uint8_t* wq, const float* ws,
              void* y, void* work, void* stream) {
    if (!x || !wq || !ws || !y) return Q4_ERR_NULL;
    const int st = check_x(M, K, xdtype, x, x_stride);
    if (st) return st;
    if (!size_ok(N, K) || !product_ok(M, N)) return Q4_ERR_DIM;
    if (!work) return Q4_ERR_NULL;  // after the sizes: those that are refused have a workspace of 0 bytes
    if (!aligned(wq, 16) || !aligned(ws, 4) || !aligned(y, 16) || !aligned(work, 16)) return Q4_ERR_ALIGN;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool bf16 = xdtype == Q4_DT_BF16;
    if (q4::f8_linear_fused(M, K, bf16, x, x_stride))
        return hip_status(q4::launch_f8_linear_fused(M, K, N, bf16, x, x_stride, wq, ws, y, s));
    uint8_t* xq = static_cast<uint8_t*>(work);
    float* xs = reinterpret_cast<float*>(xq + codes_bytes(M, K));
    const hipError_t e = q4::launch_f8_quantize_rows(M, K, bf16, x, x_stride, xq, xs, s);
    if (e != hipSuccess) return Q4_ERR_HIP;
    return hip_status(q4::launch_f8_gemm(M, N, up128(K) / 128, bf16, xq, xs, wq, ws, y, s));
}

// The workspace holds the codes and scales of dy by rows (for dx), and of dy and x by columns (for dw).
size_t f8_linear_backward_work_bytes(int M, int K, int N) {
    if (!size_ok(M, K) || !size_ok(M, N) || !size_ok(N, K) || !size_ok(K, M) || !size_ok(N, M) || !size_ok(K, N) ||
        !product_ok(M, K) || !product_ok(N, K))
        return 0;
    return codes_bytes(M, N) + scales_bytes(M, N) + codes_bytes(N, M) + scales_bytes(N, M) + codes_bytes(K, M) +
           scales_bytes(K, M);
}

int f8_linear_backward(int M, int K, int N, int dtype, const void* dy, long long dy_stride, const void* x,
                       long long x_stride, const uint8_t* wqt, const float* wst, void* dx, int dwtype, void* dw,
                       void* work, void* stream) {
    if (!dy || (!dx && !dw) || (dx && (!wqt || !wst)) || (dw && !x)) return Q4_ERR_NULL;
    if (dw && !type_ok(dwtype)) return Q4_ERR_FORMAT;
    int st = check_x(M, N, dtype, dy, dy_stride);
    if (st) return st;
    if (dw && (st = check_x(M, K, dtype, x, x_stride))) return st;
    if (!f8_linear_backward_work_bytes(M, K, N)) return Q4_ERR_DIM;
    if (!work) return Q4_ERR_NULL;
    if (!aligned(dx, 16) || !aligned(dw, 16) || !aligned(wqt, 16) || !aligned(wst, 4) || !aligned(work, 16))
        return Q4_ERR_ALIGN;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool bf16 = dtype == Q4_DT_BF16;
    uint8_t* dyq = static_cast<uint8_t*>(work);
    float* dys = reinterpret_cast<float*>(dyq + codes_bytes(M, N));
    uint8_t* dyt = reinterpret_cast<uint8_t*>(dys) + scales_bytes(M, N);
    float* dyts = reinterpret_cast<float*>(dyt + codes_bytes(N, M));
    uint8_t* xt = reinterpret_cast<uint8_t*>(dyts) + scales_bytes(N, M);
    float* xts = reinterpret_cast<float*>(xt + codes_bytes(K, M));
    if (q4::launch_f8_quantize_backward(M, K, N, bf16, dy, dy_stride, x, x_stride, dyq, dys, dyt, dyts, xt, xts,
                                        dx != nullptr, dw != nullptr, s) != hipSuccess)
        return Q4_ERR_HIP;
    if (dx && q4::launch_f8_gemm(M, K, up128(N) / 128, bf16, dyq, dys, wqt, wst, dx, s) != hipSuccess)
        return Q4_ERR_HIP;
    if (dw && q4::launch_f8_gemm_rowscales(N, K, up128(M) / 128, dwtype == Q4_DT_BF16, dyt, dyts, xt, xts, dw, s) !=
                  hipSuccess)
        return Q4_ERR_HIP;
    return Q4_OK;
}

}  // extern "C"
