// Internal interface of the orthogonalised updates (include/sgemm_ortho.h).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "experts.h"

namespace gb300 {

constexpr int kOrthoMostChunks = 256;  // row chunks of a matrix in the sums of squares

// Preparation: sums of squares, then X / (norm + eps) as two f16 planes.
struct OrthoPrep {
    const void* G;
    long long ldg, sg;
    int E, rows, cols;
    int vec;             // G's rows begin on 16 bytes
    double* part;        // E x chunks
    int chunks, per;     // row chunks a matrix, and rows of one
    double eps;
    int* shift;          // of each matrix: the power of two that its X is held times besides
    uint16_t* hi;        // planes of E x rows x pitch; `plane` elements apart
    long long pitch, plane;
    int* zero;           // counters to set to 0
    long long zeros;
};
int ortho_prepare(const OrthoPrep& p, int type, cudaStream_t s);

namespace detail {

struct DeviceState;
struct OrthoCall {
    const void* G;
    long long ldg, sg;
    void* out;
    long long ldo, so;
    int type, E, M, N, steps;
    int parts;  // f16 values that stand for an operand in the products: 2, or 1 (bf16 alone)
    float a, b, c;
    int growth;  // |p(s) / s| of the polynomial is at most 2^growth
    double eps;
    void* workspace;
};
// The workspace's parts, in bytes from its beginning.
struct OrthoLayout {
    int chunks, per, panels;       // of the preparation and of the counters
    long long pitch, square_pitch;  // elements a row of X's planes and of A's
    long long part, done, shift, d, e, a, p, x[2], bytes;
};
OrthoLayout ortho_layout(int E, int M, int N, int steps, int parts);
int orthogonalize(const OrthoCall& c, DeviceState& st, cudaStream_t s);
// The most matrices of a call: the small form numbers the CTAs of their clusters, up to 16 each, in 31 bits.
constexpr int kOrthoMostMatrices = 0x7fffffff / 16;
// Whether every device takes the call in its small form, which needs no workspace.
inline bool ortho_always_small(int M, int N) {
    return (M < N ? M : N) <= 128 && (M < N ? N : M) <= 8 * 256;
}
// A short side of up to 128 (ortho_small.cu); SGEMM_ERR_UNSUPPORTED: not one of these.
int ortho_small_set_up(int* most_ctas);
int ortho_small(const OrthoCall& c, const DeviceState& st, cudaStream_t s);

}  // namespace detail
}  // namespace gb300
