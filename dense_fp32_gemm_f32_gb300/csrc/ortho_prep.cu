// Preparation of an orthogonalised update: the norm of each matrix, and X = G /
// (norm + eps) as the products take it (ortho_tc.cuh): 2^13 X in two f16 planes,
// hi = f16(2^13 X) and lo = f16(2^13 X - hi), together 22 bits.  Bound by
// bytes: G is read twice, the planes written once.
// The parts of a matrix's sum are added in one order, so that results do not
// depend on timing.
#include "../../include/sgemm_ortho.h"
#include "experts_groups.cuh"
#include "ortho.h"
#include "ortho_load.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kPrepThreads = 256, kPrepLoads = 4;  // (8 values a load)

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
    const int n = max(rows, 0) * octs;
    for (int i = threadIdx.x; i < n; i += kPrepLoads * kPrepThreads) {
        float v[kPrepLoads][8];
        load_octs(G + r0 * p.ldg, p.ldg, i, kPrepThreads, octs, p.cols, n, p.vec && p.cols % 8 == 0, p.vec, v);
        sum += squares(v);
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
    const double norm = sqrt(cta_sum(mine, scratch));
    const int shift = ortho_shift(norm, p.eps);
    if (chunk == 0 && threadIdx.x == 0) p.shift[e] = shift;
    const OrthoScale scale(norm + p.eps, shift);
    const int octs = (p.cols + 7) / 8;
    const int r0 = chunk * p.per, rows = min(p.per, p.rows - r0);
    const T* G = static_cast<const T*>(p.G) + e * p.sg;
    const int n = max(rows, 0) * octs;
    uint16_t* const to = p.hi + (static_cast<long long>(e) * p.rows + r0) * p.pitch;
    for (int i = threadIdx.x; i < n; i += kPrepLoads * kPrepThreads) {
        float v[kPrepLoads][8];
        load_octs(G + r0 * p.ldg, p.ldg, i, kPrepThreads, octs, p.cols, n, p.vec && p.cols % 8 == 0, p.vec, v);
#pragma unroll
        for (int u = 0; u < kPrepLoads; ++u) {
            const int at = i + u * kPrepThreads, r = at / octs, c = (at - r * octs) * 8;
            if (at >= n) break;
            uint4 hi, lo;
            scale.split(v[u], hi, lo);
            uint16_t* const d = to + r * p.pitch + c;
            *reinterpret_cast<uint4*>(d) = hi;
            *reinterpret_cast<uint4*>(d + p.plane) = lo;
        }
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
