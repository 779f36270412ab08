// Rows of tokens to their places by expert, and back (include/sgemm_routing.h).
// Bound by bytes: every row of the tokens once and every row of the choices
// once (twice for the gradient of a combination).  A thread takes a vector of
// a token's columns (16 bytes where the rows' alignment allows) and goes
// through the token's choices, so that the token's row stays in a register
// and each choice's row is one stream of whole lines.
#include "../../include/sgemm_routing.h"
#include "experts_groups.cuh"
#include "ptx.cuh"
#include "routing.h"

namespace gb300 {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRowsThreads = 256;

// N elements of T as one access of N * sizeof(T) bytes (at most 16).
template <typename T, int N>
struct alignas(N * sizeof(T)) Vec {
    T v[N];
};

__device__ __forceinline__ int slot_of(const RowsParams& p, long long i) {
    const int s = __ldg(p.slots + i);
    return s >= 0 && s < p.R ? s : -1;
}

// Zeros to the rows from *used on, `worker` of `workers` threads.
template <typename T, int N>
__device__ __forceinline__ void zero_unused(const RowsParams& p, long long worker, long long workers, int nvec) {
    const int used = min(max(__ldg(p.used), 0), p.R);
    const long long n = static_cast<long long>(p.R - used) * nvec;
    for (long long i = worker; i < n; i += workers) {
        const long long r = i / nvec;
        const int c = static_cast<int>(i - r * nvec) * N;
        T* o = static_cast<T*>(p.out) + (used + r) * p.ldo + c;
        if (c + N <= p.H) {
            Vec<T, N> z;
#pragma unroll
            for (int j = 0; j < N; ++j) z.v[j] = from_f32<T>(0.f);
            *reinterpret_cast<Vec<T, N>*>(o) = z;
        } else {
            for (int j = 0; c + j < p.H; ++j) o[j] = from_f32<T>(0.f);
        }
    }
}

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T* p, int left) {
    if (left >= N) return *reinterpret_cast<const Vec<T, N>*>(p);
    Vec<T, N> x;
#pragma unroll
    for (int j = 0; j < N; ++j) x.v[j] = j < left ? p[j] : from_f32<T>(0.f);
    return x;
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, N>& x, int left) {
    if (left >= N) {
        *reinterpret_cast<Vec<T, N>*>(p) = x;
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < left) p[j] = x.v[j];
    }
}

template <typename T, int N>
__global__ void __launch_bounds__(kRowsThreads) spread_kernel(const RowsParams p, uint32_t nvec) {
    const long long id = static_cast<long long>(blockIdx.x) * kRowsThreads + threadIdx.x;
    const long long t = id / nvec;
    if (t < p.T) {
        const int c = static_cast<int>(id - t * nvec) * N, left = p.H - c;
        const Vec<T, N> x = load_vec<T, N>(static_cast<const T*>(p.X) + t * p.ldx + c, left);
        for (int j = 0; j < p.k; ++j) {
            const int s = slot_of(p, t * p.k + j);
            if (s >= 0) store_vec<T, N>(static_cast<T*>(p.out) + s * p.ldo + c, x, left);
        }
    }
    zero_unused<T, N>(p, id, static_cast<long long>(gridDim.x) * kRowsThreads, nvec);
}

template <typename T, int N>
__global__ void __launch_bounds__(kRowsThreads) combine_kernel(const RowsParams p, uint32_t nvec) {
    const long long id = static_cast<long long>(blockIdx.x) * kRowsThreads + threadIdx.x;
    const long long t = id / nvec;
    if (t >= p.T) return;
    const int c = static_cast<int>(id - t * nvec) * N, left = p.H - c;
    float sum[N] = {};
#pragma unroll 4
    for (int j = 0; j < p.k; ++j) {
        const int s = slot_of(p, t * p.k + j);
        if (s >= 0) {
            const float w = p.weights ? __ldg(p.weights + t * p.k + j) : 1.f;
            const Vec<T, N> y = load_vec<T, N>(static_cast<const T*>(p.Y) + s * p.ldy + c, left);
#pragma unroll
            for (int i = 0; i < N; ++i) sum[i] = fmaf(w, to_f32(y.v[i]), sum[i]);
        }
    }
    Vec<T, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.v[i] = from_f32<T>(sum[i]);
    store_vec<T, N>(static_cast<T*>(p.out) + t * p.ldo + c, o, left);
}

// A token to `group` threads (a power of two, 32 to 256), choices 8 at a time.
template <typename T, int N>
__global__ void __launch_bounds__(kRowsThreads) combine_grad_kernel(const RowsParams p, int nvec, int group) {
    constexpr int kBatch = 8;
    __shared__ float part[kRowsThreads / 32][kBatch];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int member = threadIdx.x & (group - 1);
    const long long t = static_cast<long long>(blockIdx.x) * (kRowsThreads / group) + threadIdx.x / group;
    const bool there = t < p.T;
    for (int j0 = 0; j0 < p.k; j0 += kBatch) {
        int slot[kBatch];
        float w[kBatch], dot[kBatch] = {};
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const bool in = there && j0 + b < p.k;
            slot[b] = in ? slot_of(p, t * p.k + j0 + b) : -1;
            w[b] = in && p.weights ? __ldg(p.weights + t * p.k + j0 + b) : 1.f;
        }
        if (there) {
            for (int v = member; v < nvec; v += group) {
                const int c = v * N, left = p.H - c;
                const Vec<T, N> d = load_vec<T, N>(static_cast<const T*>(p.X) + t * p.ldx + c, left);
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    if (slot[b] < 0) continue;
                    if (p.dweights) {
                        const Vec<T, N> y = load_vec<T, N>(static_cast<const T*>(p.Y) + slot[b] * p.ldy + c, left);
#pragma unroll
                        for (int i = 0; i < N; ++i) dot[b] = fmaf(to_f32(d.v[i]), to_f32(y.v[i]), dot[b]);
                    }
                    if (p.out) {
                        Vec<T, N> o;
#pragma unroll
                        for (int i = 0; i < N; ++i) o.v[i] = from_f32<T>(w[b] * to_f32(d.v[i]));
                        store_vec<T, N>(static_cast<T*>(p.out) + slot[b] * p.ldo + c, o, left);
                    }
                }
            }
        }
        if (p.dweights) {
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
#pragma unroll
                for (int s = 16; s; s /= 2) dot[b] += __shfl_xor_sync(kAll, dot[b], s);
            if (group > 32) {
                if (lane == 0) {
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) part[warp][b] = dot[b];
                }
                __syncthreads();
                if (member < kBatch && there && j0 + member < p.k) {
                    float sum = 0.f;
                    for (int q = 0; q < group / 32; ++q) sum += part[warp + q][member];
                    p.dweights[t * p.k + j0 + member] = sum;
                }
                __syncthreads();
            } else if (there) {
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
                    if (lane == b && j0 + b < p.k) p.dweights[t * p.k + j0 + b] = dot[b];
            }
        }
    }
    if (p.out)
        zero_unused<T, N>(p, static_cast<long long>(blockIdx.x) * kRowsThreads + threadIdx.x,
                          static_cast<long long>(gridDim.x) * kRowsThreads, nvec);
}

// f(T(), integral_constant<vector length>).
template <typename F>
int by_type_and_vec(int type, int vec, F f) {
    if (type == SGEMM_TYPE_F32) {
        if (vec == 4) return f(0.f, std::integral_constant<int, 4>());
        if (vec == 2) return f(0.f, std::integral_constant<int, 2>());
        return f(0.f, std::integral_constant<int, 1>());
    }
    auto half = [&](auto zero) {
        if (vec == 8) return f(zero, std::integral_constant<int, 8>());
        if (vec == 4) return f(zero, std::integral_constant<int, 4>());
        if (vec == 2) return f(zero, std::integral_constant<int, 2>());
        return f(zero, std::integral_constant<int, 1>());
    };
    return type == SGEMM_TYPE_BF16 ? half(__nv_bfloat16()) : half(__half());
}

int launched() { return cudaGetLastError() == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA; }

// CTAs for `threads` threads; -1 if a grid cannot hold them.
long long ctas_for(long long threads) {
    const long long n = (threads + kRowsThreads - 1) / kRowsThreads;
    return n <= 0x7fffffffll ? n : -1;
}

}  // namespace

int rows_spread(const RowsParams& p, int type, int sms, cudaStream_t s) {
    const uint32_t nvec = static_cast<uint32_t>((p.H + p.vec - 1) / p.vec);
    const long long n = ctas_for(static_cast<long long>(p.T) * nvec);
    if (n < 0) return SGEMM_ERR_INVALID_ARG;
    const unsigned ctas = static_cast<unsigned>(n > sms ? n : sms);  // (the rows to zero are shared among all)
    return by_type_and_vec(type, p.vec, [&](auto zero, auto vec) {
        spread_kernel<decltype(zero), decltype(vec)::value><<<ctas, kRowsThreads, 0, s>>>(p, nvec);
        return launched();
    });
}

int rows_combine(const RowsParams& p, int type, int sms, cudaStream_t s) {
    (void)sms;
    const uint32_t nvec = static_cast<uint32_t>((p.H + p.vec - 1) / p.vec);
    const long long n = ctas_for(static_cast<long long>(p.T) * nvec);
    if (n < 0) return SGEMM_ERR_INVALID_ARG;
    return by_type_and_vec(type, p.vec, [&](auto zero, auto vec) {
        combine_kernel<decltype(zero), decltype(vec)::value><<<static_cast<unsigned>(n), kRowsThreads, 0, s>>>(p, nvec);
        return launched();
    });
}

int rows_combine_grad(const RowsParams& p, int type, int sms, cudaStream_t s) {
    const int nvec = (p.H + p.vec - 1) / p.vec;
    // Threads a token: all that have a vector, unless there are tokens enough.
    int group = kRowsThreads;
    while (group > 32 && (group / 2 >= nvec || static_cast<long long>(p.T) * group > 2048ll * 8 * sms)) group /= 2;
    const long long n = ctas_for(static_cast<long long>(p.T) * group);
    if (n < 0) return SGEMM_ERR_INVALID_ARG;
    const unsigned ctas = static_cast<unsigned>(p.out && n < sms ? sms : n);
    return by_type_and_vec(type, p.vec, [&](auto zero, auto vec) {
        combine_grad_kernel<decltype(zero), decltype(vec)::value><<<ctas, kRowsThreads, 0, s>>>(p, nvec, group);
        return launched();
    });
}

}  // namespace gb300
