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
    float a, b, c;
    double eps;
};
int orthogonalize(const OrthoCall& c, int dev, DeviceState& st, cudaStream_t s);
// A short side of up to 128 (ortho_small.cu); SGEMM_ERR_UNSUPPORTED: not one of these.
int ortho_small_set_up(int* most_ctas);
int ortho_small(const OrthoCall& c, const DeviceState& st, cudaStream_t s);

}  // namespace detail
}  // namespace gb300
