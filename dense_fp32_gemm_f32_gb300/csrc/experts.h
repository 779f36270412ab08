// Internal interface of the grouped products and the MXFP4 operators
// (include/sgemm_experts.h): kernel parameters and launch functions.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace gb300 {

// One operand copied for the tensor maps (experts_pack.cu): `count` matrices
// of rows x cols at src (`ld` elements a row, `se` a matrix) to dst, rows of
// dld elements (a multiple of 8) one after the other; float32 to three bf16
// planes one after the other.  dst null: nothing to do.  offsets: matrix e is
// expert e's, and one without rows need not be copied (T: the rows in all).
struct PackJob {
    const void* src;
    long long count, rows, ld, se;
    int cols;
    void* dst;
    long long dld;
    const int* offsets;
    int T;
    long long each;  // rows of a matrix where `rows` holds all (set by experts_pack)
};
int experts_pack(const PackJob& a, const PackJob& b, bool f32, cudaStream_t s);

// MXFP4 quantisation and its inverse (mxfp4.cu).
struct QuantParams {
    const void* X;
    long long ldx, sx;
    void* Y;
    long long ldy, sy;
    uint8_t* codes;
    uint8_t* scales;
    const uint8_t* codes_in;
    const uint8_t* scales_in;
    const int* offsets;  // null: no groups
    int E, batch, rows, K;
};
int mxfp4_quantize(const QuantParams& p, int type, cudaStream_t s);
int mxfp4_dequantize(const QuantParams& p, int type, cudaStream_t s);

namespace detail {

// `count` matrices of rows x cols, `ld` elements a row, `se` a matrix.
struct MatrixArg {
    const void* p;
    long long count, rows, cols, ld, se;
};

// A grouped product as the tensor-core kernels take it (experts_tc.cuh):
// forward: a = the weights (F the output's columns, K the contraction), b = X;
// weight gradient: a = X (F its columns), b = dY (C its columns).
struct GroupedCall {
    MatrixArg a, b;
    bool wgrad, a_mn;  // a_mn: the weights' contiguous dimension is F
    int type, out_type;
    int T, E, F, C, K;
    const int* offsets;
    void* out;
    long long ldo, so;
};

// An MXFP4 product as mxfp4_tc.cuh takes it: rows X (T x K), weights W (E
// matrices N x K); offsets null: one matrix.
struct Mxfp4Call {
    const uint8_t *X, *x_scales, *W, *w_scales;
    long long x_blocks;  // row blocks of X's scales
    int out_type, T, E, N, K;
    const int* offsets;
    void* out;
    long long ldo;
};

// Bytes (2 .. 16) that the rows of an output of `size`-byte elements are
// aligned to.
inline int row_alignment(const void* out, int size, long long ld, long long stride) {
    const unsigned long long bits = reinterpret_cast<uintptr_t>(out) | size * ld | size * stride | 16;
    return static_cast<int>(bits & (~bits + 1));
}

// CTAs that share a tile's contraction where `tiles` (at most) leave half of the
// SMs idle: as many as keep every cluster on one tile, with parts of `least`
// or more.
inline int split_parts(long long tiles, int K, int least, int sms) {
    int ks = 1;
    while (ks < 8 && 2 * ks * tiles <= sms && K >= 2 * ks * least) ks *= 2;
    return ks;
}

struct DeviceState;
int mxfp4_tc_set_up();
int mxfp4_tc(const Mxfp4Call& c, const DeviceState& st, cudaStream_t s);
int experts_tc_set_up(DeviceState& st);
int grouped_tc(const GroupedCall& c, int dev, DeviceState& st, cudaStream_t s);
// Forward products of float32 operands with few rows a group (experts_few.cu).
int experts_few_set_up();
int grouped_few(const GroupedCall& c, const DeviceState& st, cudaStream_t s);

}  // namespace detail
}  // namespace gb300
