// The entry points of include/sgemm_experts.h: argument checks, operand
// layouts and the choice of kernel.
#include "../../include/sgemm_experts.h"
#include "api_internal.h"
#include "experts.h"

using namespace gb300;
using namespace gb300::detail;

namespace {

bool type_ok(int t) { return t == SGEMM_TYPE_F32 || t == SGEMM_TYPE_BF16 || t == SGEMM_TYPE_F16; }
int type_bytes(int t) { return t == SGEMM_TYPE_F32 ? 4 : 2; }

// `count` matrices of rows x cols elements of `size` bytes, `ld` elements a
// row and `stride` elements a matrix.
struct View {
    const void* p;
    int64_t count, rows, cols, ld, stride;
    int size;

    bool empty() const { return count == 0 || rows == 0 || cols == 0; }
    size_t bytes() const {
        return empty() ? 0 : static_cast<size_t>(((count - 1) * stride + (rows - 1) * ld + cols) * size);
    }
    // Rows do not overlap, matrices do not overlap, the pointer is aligned,
    // and the array's size fits its type.
    bool ok(uintptr_t align) const {
        if (empty()) return true;
        if (!p || (reinterpret_cast<uintptr_t>(p) & (align - 1))) return false;
        if (rows > 1 && ld < cols) return false;
        constexpr int64_t most = int64_t{1} << 56;
        if (ld > most / rows / size || (count > 1 && stride > most / count / size)) return false;
        return count <= 1 || stride >= (rows - 1) * ld + cols;
    }
};

bool overlap(const View& a, const View& b) { return ranges_overlap(a.p, a.bytes(), b.p, b.bytes()); }

bool offsets_ok(const int* offsets) { return offsets && !(reinterpret_cast<uintptr_t>(offsets) & 3); }

int64_t blocks32(int64_t k) { return (k + 31) / 32; }
int64_t blocks128(int64_t n) { return (n + 127) / 128; }

View codes_view(const uint8_t* p, int64_t count, int64_t rows, int64_t K) {
    return {p, count, rows, 16 * blocks32(K), 16 * blocks32(K), rows * 16 * blocks32(K), 1};
}
View scales_view(const uint8_t* p, int64_t count, int64_t row_blocks, int64_t K) {
    return {p, count, row_blocks, 512 * blocks128(K), 512 * blocks128(K), row_blocks * 512 * blocks128(K), 1};
}
// Row blocks of T rows grouped by E experts, at most.
int64_t grouped_blocks(int64_t T, int64_t E) { return (T + 127 * std::min(T, E)) / 128; }

// Zeros to `count` matrices of rows x cols: in one operation, unless both the rows
// and the matrices lie apart.
int zero_rows(void* p, int64_t count, int64_t rows, int64_t cols, int64_t ld, int64_t stride, int size,
              cudaStream_t s) {
    if (count > 1 && stride == rows * ld) {  // (rows of one matrix)
        rows *= count;
        count = 1;
    } else if (count > 1 && (ld == cols || rows == 1)) {  // (a matrix is a row)
        cols *= rows;
        rows = count;
        ld = stride;
        count = 1;
    }
    for (int64_t e = 0; e < count; ++e)
        if (rows > 0 && cols > 0 &&
            cudaMemset2DAsync(static_cast<char*>(p) + e * stride * size, ld * size, 0, cols * size, rows, s) !=
                cudaSuccess) {
            (void)cudaGetLastError();
            return SGEMM_ERR_CUDA;
        }
    return SGEMM_OK;
}

// Largest dimension and number of experts that the kernels number with ints.
constexpr int kMost = 1 << 30;

}  // namespace

extern "C" {

int sgemm_grouped(int type, int transw, int T, int E, int N, int K, const void* X, int64_t ldx, const void* W,
                  int64_t ldw, int64_t stride_w, const int* offsets, void* Y, int64_t ldy, void* stream) {
    if (!type_ok(type) || (transw != 0 && transw != 1)) return SGEMM_ERR_INVALID_ARG;
    if (T < 0 || E < 0 || N < 0 || K < 0 || T > kMost || E > kMost || N > kMost || K > kMost)
        return SGEMM_ERR_INVALID_ARG;
    const int size = type_bytes(type);
    const View x{X, 1, T, K, ldx, 0, size}, y{Y, 1, T, N, ldy, 0, size};
    const View w{W, E, transw ? N : K, transw ? K : N, ldw, stride_w, size};
    if (!x.ok(size) || !w.ok(size) || !y.ok(size) || !offsets_ok(offsets) || overlap(y, x) || overlap(y, w))
        return SGEMM_ERR_INVALID_ARG;
    if (y.empty()) return SGEMM_OK;
    int dev = 0;
    DeviceState* st = nullptr;
    const int rc = experts_device(&dev, &st);
    if (rc != SGEMM_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (E == 0 || K == 0) return zero_rows(Y, 1, T, N, ldy, 0, size, s);
    GroupedCall c = {};
    c.a = {W, E, transw ? N : K, transw ? K : N, ldw, stride_w};
    c.b = {X, 1, T, K, ldx, 0};
    c.a_mn = !transw;
    c.type = c.out_type = type;
    c.T = T, c.E = E, c.F = N, c.K = K;
    c.offsets = offsets;
    c.out = Y, c.ldo = ldy;
    return grouped_tc(c, dev, *st, s);
}

int sgemm_grouped_wgrad(int type, int out_type, int T, int E, int K, int N, const void* X, int64_t ldx,
                        const void* dY, int64_t lddy, const int* offsets, void* dW, int64_t lddw, int64_t stride_dw,
                        void* stream) {
    if (!type_ok(type) || (out_type != type && out_type != SGEMM_TYPE_F32)) return SGEMM_ERR_INVALID_ARG;
    if (T < 0 || E < 0 || N < 0 || K < 0 || T > kMost || E > kMost || N > kMost || K > kMost)
        return SGEMM_ERR_INVALID_ARG;
    const int size = type_bytes(type), osize = type_bytes(out_type);
    const View x{X, 1, T, K, ldx, 0, size}, dy{dY, 1, T, N, lddy, 0, size};
    const View dw{dW, E, K, N, lddw, stride_dw, osize};
    if (!x.ok(size) || !dy.ok(size) || !dw.ok(osize) || !offsets_ok(offsets) || overlap(dw, x) || overlap(dw, dy))
        return SGEMM_ERR_INVALID_ARG;
    if (dw.empty()) return SGEMM_OK;
    int dev = 0;
    DeviceState* st = nullptr;
    const int rc = experts_device(&dev, &st);
    if (rc != SGEMM_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) return zero_rows(dW, E, K, N, lddw, stride_dw, osize, s);
    GroupedCall c = {};
    c.a = {X, 1, T, K, ldx, 0};
    c.b = {dY, 1, T, N, lddy, 0};
    c.wgrad = c.a_mn = true;
    c.type = type, c.out_type = out_type;
    c.T = T, c.E = E, c.F = K, c.C = N;
    c.offsets = offsets;
    c.out = dW, c.ldo = lddw, c.so = stride_dw;
    return grouped_tc(c, dev, *st, s);
}

static int quant_check(int type, int batch, int rows, int K, const View& x, int E, const int* offsets,
                       const uint8_t* codes, const uint8_t* scales) {
    if (!type_ok(type) || batch < 0 || rows < 0 || K < 0 || E < 0) return SGEMM_ERR_INVALID_ARG;
    if (batch > kMost || rows > kMost || K > kMost || E > kMost) return SGEMM_ERR_INVALID_ARG;
    if (offsets && (batch != 1 || !offsets_ok(offsets))) return SGEMM_ERR_INVALID_ARG;
    if (!offsets && E != 0) return SGEMM_ERR_INVALID_ARG;
    const View c = codes_view(codes, batch, rows, K);
    const View sc = scales_view(scales, batch, offsets ? grouped_blocks(rows, E) : blocks128(rows), K);
    if (!x.ok(x.size) || !c.ok(16) || !sc.ok(16)) return SGEMM_ERR_INVALID_ARG;
    if (overlap(x, c) || overlap(x, sc) || overlap(c, sc)) return SGEMM_ERR_INVALID_ARG;
    return SGEMM_OK;
}

int sgemm_mxfp4_quantize(int type, int batch, int rows, int K, const void* X, int64_t ldx, int64_t stride_x, int E,
                         const int* offsets, uint8_t* codes, uint8_t* scales, void* stream) {
    const View x{X, batch, rows, K, ldx, stride_x, type_bytes(type)};
    int rc = quant_check(type, batch, rows, K, x, E, offsets, codes, scales);
    if (rc != SGEMM_OK || x.empty()) return rc;
    int dev = 0;
    DeviceState* st = nullptr;
    rc = current_device(&dev, &st);
    if (rc != SGEMM_OK) return rc;
    QuantParams p = {};
    p.X = X, p.ldx = ldx, p.sx = stride_x;
    p.codes = codes, p.scales = scales;
    p.offsets = offsets, p.E = E, p.batch = batch, p.rows = rows, p.K = K;
    return mxfp4_quantize(p, type, static_cast<cudaStream_t>(stream));
}

int sgemm_mxfp4_dequantize(int type, int batch, int rows, int K, const uint8_t* codes, const uint8_t* scales, int E,
                           const int* offsets, void* Y, int64_t ldy, int64_t stride_y, void* stream) {
    const View y{Y, batch, rows, K, ldy, stride_y, type_bytes(type)};
    int rc = quant_check(type, batch, rows, K, y, E, offsets, codes, scales);
    if (rc != SGEMM_OK || y.empty()) return rc;
    int dev = 0;
    DeviceState* st = nullptr;
    rc = current_device(&dev, &st);
    if (rc != SGEMM_OK) return rc;
    QuantParams p = {};
    p.Y = Y, p.ldy = ldy, p.sy = stride_y;
    p.codes_in = codes, p.scales_in = scales;
    p.offsets = offsets, p.E = E, p.batch = batch, p.rows = rows, p.K = K;
    return mxfp4_dequantize(p, type, static_cast<cudaStream_t>(stream));
}

static int mxfp4_product(int out_type, int T, int E, int N, int K, const uint8_t* X, const uint8_t* x_scales,
                         const uint8_t* W, const uint8_t* w_scales, const int* offsets, void* Y, int64_t ldy,
                         void* stream) {
    if (!type_ok(out_type) || T < 0 || E < 0 || N < 0 || K < 0 || T > kMost || E > kMost || N > kMost || K > kMost)
        return SGEMM_ERR_INVALID_ARG;
    const int size = type_bytes(out_type);
    const View x = codes_view(X, 1, T, K), w = codes_view(W, E, N, K), y{Y, 1, T, N, ldy, 0, size};
    const View xs = scales_view(x_scales, 1, offsets ? grouped_blocks(T, E) : blocks128(T), K);
    const View ws = scales_view(w_scales, E, blocks128(N), K);
    if (!x.ok(16) || !w.ok(16) || !xs.ok(16) || !ws.ok(16) || !y.ok(size)) return SGEMM_ERR_INVALID_ARG;
    if (overlap(y, x) || overlap(y, xs) || overlap(y, w) || overlap(y, ws)) return SGEMM_ERR_INVALID_ARG;
    if (y.empty()) return SGEMM_OK;
    int dev = 0;
    DeviceState* st = nullptr;
    const int rc = experts_device(&dev, &st);
    if (rc != SGEMM_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (E == 0 || K == 0) return zero_rows(Y, 1, T, N, ldy, 0, size, s);
    Mxfp4Call c = {X, x_scales, W, w_scales, xs.rows, out_type, T, E, N, K, offsets, Y, ldy};
    return mxfp4_tc(c, *st, s);
}

int sgemm_mxfp4(int out_type, int M, int N, int K, const uint8_t* A, const uint8_t* a_scales, const uint8_t* B,
                const uint8_t* b_scales, void* C, int64_t ldc, void* stream) {
    return mxfp4_product(out_type, M, 1, N, K, A, a_scales, B, b_scales, nullptr, C, ldc, stream);
}

int sgemm_mxfp4_grouped(int out_type, int T, int E, int N, int K, const uint8_t* X, const uint8_t* x_scales,
                        const uint8_t* W, const uint8_t* w_scales, const int* offsets, void* Y, int64_t ldy,
                        void* stream) {
    if (!offsets_ok(offsets)) return SGEMM_ERR_INVALID_ARG;
    return mxfp4_product(out_type, T, E, N, K, X, x_scales, W, w_scales, offsets, Y, ldy, stream);
}

}  // extern "C"
