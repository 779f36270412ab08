// Internal interface of the grouped products and the MXFP4 operators
// (include/sgemm_experts.h): kernel parameters and launch functions.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace gb300 {

// One operand of a product in HBM, element (row, k) of matrix e.
struct StridedOperand {
    const void* p;
    long long se, sr, sk;  // strides in elements: matrix, row, contraction
};

// MXFP4 operand: codes (rows of `pitch` bytes) and scale blocks.
struct Mxfp4Operand {
    const uint8_t* codes;
    const uint8_t* scales;
    long long codes_e, scales_e;  // bytes between matrices
    int pitch;                    // bytes per row of codes
    int kq;                       // scale blocks per row of blocks
};

// The simple kernels' launch (experts_simple.cu).  mode: rows of the first
// operand grouped (forward), or the contraction grouped (weight gradient).
struct SimpleParams {
    StridedOperand A, B;    // A: (rows or the output's rows) x k, B: (columns) x k
    Mxfp4Operand qA, qB;
    const int* offsets;     // null: one group of all T rows
    int T, E;
    int R, N, K;            // weight gradient: output rows R; forward: R unused
    void* out;
    long long ldo, so;      // output row pitch; matrix stride (weight gradient)
};
int simple_forward(const SimpleParams& p, int type, cudaStream_t s);
int simple_wgrad(const SimpleParams& p, int type, int out_type, cudaStream_t s);
int simple_mxfp4(const SimpleParams& p, int out_type, cudaStream_t s);

// One operand copied for the tensor maps (experts_pack.cu): `count` matrices
// of rows x cols at src (`ld` elements a row, `se` a matrix) to dst, rows of
// dld elements (a multiple of 8) one after the other; float32 to three bf16
// planes one after the other.  dst null: nothing to do.
struct PackJob {
    const void* src;
    long long count, rows, ld, se;
    int cols;
    void* dst;
    long long dld;
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
// weight gradient: a = dY (F its columns), b = X (C its columns).
struct GroupedCall {
    MatrixArg a, b;
    bool wgrad, a_mn;  // a_mn: the weights' contiguous dimension is F
    int type, out_type;
    int T, E, F, C, K;
    const int* offsets;
    void* out;
    long long ldo, so;
};

struct DeviceState;
int experts_tc_set_up(DeviceState& st);
int grouped_tc(const GroupedCall& c, int dev, DeviceState& st, cudaStream_t s);

}  // namespace detail
}  // namespace gb300
