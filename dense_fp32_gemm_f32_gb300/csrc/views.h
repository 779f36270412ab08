// Argument checks that the entry points of typed operands share
// (api_experts.cu, api_routing.cu, api_ortho.cu).
#pragma once

#include "../../include/sgemm_experts.h"
#include "api_internal.h"

namespace gb300 {
namespace detail {

inline bool type_ok(int t) { return t == SGEMM_TYPE_F32 || t == SGEMM_TYPE_BF16 || t == SGEMM_TYPE_F16; }
inline int type_bytes(int t) { return t == SGEMM_TYPE_F32 ? 4 : 2; }

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

inline bool overlap(const View& a, const View& b) { return ranges_overlap(a.p, a.bytes(), b.p, b.bytes()); }

inline bool offsets_ok(const int* offsets) { return offsets && !(reinterpret_cast<uintptr_t>(offsets) & 3); }

// Zeros to `count` matrices of rows x cols: in one operation, unless both the rows
// and the matrices lie apart.
inline int zero_rows(void* p, int64_t count, int64_t rows, int64_t cols, int64_t ld, int64_t stride, int size,
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

}  // namespace detail
}  // namespace gb300
