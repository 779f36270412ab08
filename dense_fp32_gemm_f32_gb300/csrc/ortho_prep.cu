// Preparation of an orthogonalised update: the norm of each matrix, and X = G /
// (norm + eps) as the products take it (ortho_tc.cuh): 2^13 X in two f16 planes,
// hi = f16(2^13 X) and lo = f16(2^13 X - hi), together 22 bits.  Bound by
// bytes: G is read twice, the planes written once.
//
// Sums of squares.  A thread scales its values by a power of two that brings
// its largest near 1, sums their squares in float32, and adds the sum, scaled
// back, to others in 64 bits: no square overflows or vanishes.  The parts of a
// matrix are added in one order, so that results do not depend on timing.
#include "../../include/sgemm_ortho.h"
#include "experts_groups.cuh"
#include "ortho.h"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kPrepThreads = 256;

// Eight neighbouring values of a row with `left` of them there.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, bool vec, float (&v)[8]) {
    if (vec && left >= 8) {
        alignas(16) T x[8];
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
            reinterpret_cast<uint4*>(x)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f32(p[i]) : 0.f;
    }
}

// The CTA's sum of `v`, in every thread.
__device__ __forceinline__ double cta_sum(double v, double* scratch) {
#pragma unroll
    for (int d = 16; d; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kPrepThreads / 32; ++w) v += scratch[w];
    __syncthreads();
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kPrepThreads) ortho_norm_kernel(const OrthoPrep p) {
    __shared__ double scratch[kPrepThreads / 32];
    grid_dependency_launch();
    for (long long i = blockIdx.x * static_cast<long long>(kPrepThreads) + threadIdx.x; i < p.zeros;
         i += static_cast<long long>(gridDim.x) * kPrepThreads)
        p.zero[i] = 0;
    const int e = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
    const int octs = (p.cols + 7) / 8;
    const int r0 = chunk * p.per, rows = min(p.per, p.rows - r0);
    const T* G = static_cast<const T*>(p.G) + e * p.sg;
    double sum = 0;
    const long long n = static_cast<long long>(max(rows, 0)) * octs;
    for (long long i = threadIdx.x; i < n; i += kPrepThreads) {
        const int r = static_cast<int>(i / octs), c = static_cast<int>(i - static_cast<long long>(r) * octs) * 8;
        float v[8];
        load8(G + (r0 + r) * p.ldg + c, p.cols - c, p.vec, v);
        float most = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(v[j]));  // (a NaN is passed over here and summed below)
        // 2^up brings it to [1, 2) or, from below 2^-126 or above, near that
        const int up = most > 0.f ? min(126, 127 - static_cast<int>(__float_as_uint(most) >> 23)) : 0;
        const float scale = __uint_as_float(static_cast<uint32_t>(max(up, -126) + 127) << 23);
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = v[j] * scale;
            s = fmaf(x, x, s);
        }
        // (s is 0 or above 2^-50, below 2^7, and 2^-2up within a double's range)
        sum += s * __longlong_as_double(static_cast<long long>(1023 - 2 * max(up, -126)) << 52);
    }
    sum = cta_sum(sum, scratch);
    if (threadIdx.x == 0) p.part[static_cast<long long>(e) * p.chunks + chunk] = sum;
}

template <typename T>
__global__ void __launch_bounds__(kPrepThreads) ortho_split_kernel(const OrthoPrep p) {
    __shared__ double scratch[kPrepThreads / 32];
    grid_dependency_launch();
    const int e = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
    grid_dependency_wait();
    static_assert(kPrepThreads >= kOrthoMostChunks, "a part a thread");
    const double mine = threadIdx.x < p.chunks ? p.part[static_cast<long long>(e) * p.chunks + threadIdx.x] : 0.;
    // 2^13 / (norm + eps) as 2^up * factor, up a power that float32 holds and
    // the factor near 1 where it can be: X's elements stay in range between.
    const double inv = 1. / (sqrt(cta_sum(mine, scratch)) + p.eps);
    const int exponent = static_cast<int>(__double_as_longlong(inv) >> 52 & 0x7ff) - 1023;
    const int up = min(max(exponent, -126), 126);
    const float scale = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
    const float factor = static_cast<float>(inv * __longlong_as_double(static_cast<long long>(1023 - up) << 52)) * 8192.f;
    const int octs = (p.cols + 7) / 8;
    const int r0 = chunk * p.per, rows = min(p.per, p.rows - r0);
    const T* G = static_cast<const T*>(p.G) + e * p.sg;
    const long long n = static_cast<long long>(max(rows, 0)) * octs;
    for (long long i = threadIdx.x; i < n; i += kPrepThreads) {
        const int r = static_cast<int>(i / octs), c = static_cast<int>(i - static_cast<long long>(r) * octs) * 8;
        float v[8];
        load8(G + (r0 + r) * p.ldg + c, p.cols - c, p.vec, v);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = v[2 * j] * scale * factor, y = v[2 * j + 1] * scale * factor;
            const __half2 h = __floats2half2_rn(x, y);
            hi[j] = *reinterpret_cast<const uint32_t*>(&h);
            lo[j] = pair_from_f32<__half>(x - __low2float(h), y - __high2float(h));
        }
        uint16_t* d = p.hi + (static_cast<long long>(e) * p.rows + r0 + r) * p.pitch + c;
        *reinterpret_cast<uint4*>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(d + p.plane) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

template <typename T>
int prepare(const OrthoPrep& p, cudaStream_t s) {
    const unsigned ctas = static_cast<unsigned>(p.E) * static_cast<unsigned>(p.chunks);
    ortho_norm_kernel<T><<<ctas, kPrepThreads, 0, s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return SGEMM_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPrepThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, ortho_split_kernel<T>, p) != cudaSuccess) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

}  // namespace

int ortho_prepare(const OrthoPrep& p, int type, cudaStream_t s) {
    if (type == SGEMM_TYPE_F32) return prepare<float>(p, s);
    if (type == SGEMM_TYPE_BF16) return prepare<__nv_bfloat16>(p, s);
    return prepare<__half>(p, s);
}

}  // namespace gb300
