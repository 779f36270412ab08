// Rows of tokens to their places by expert, and back (include/sgemm_routing.h).
// Bound by bytes: every row of the tokens once and every row of the choices
// once (twice for the gradient of a combination).  A thread takes a vector of
// a token's columns (16 bytes where the rows' alignment allows) and goes
// through the token's choices, so that the token's row stays in a register
// and each choice's row is one stream of whole lines.
//
// Measured on GB300: 8192 tokens of 4096 bf16 to 4 experts each 51 us (6.5 TB/s); 8
// choices of 2048 combined 49 us (6.1 TB/s), and the gradient of that 97 us (5.9 TB/s; 95 without the comparison of
// every slot with the rows in use).
#include "../../include/sgemm_routing.h"
#include <algorithm>
#include <type_traits>

#include "experts_groups.cuh"
#include "ptx.cuh"
#include "routing.h"

namespace gb300 {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRowsThreads = 256;

// N elements of T as one access of N * sizeof(T) bytes (2 to 16).
template <int BYTES>
struct Word;
template <>
struct Word<16> {
    using type = uint4;
};
template <>
struct Word<8> {
    using type = uint2;
};
template <>
struct Word<4> {
    using type = uint32_t;
};
template <>
struct Word<2> {
    using type = uint16_t;
};
template <typename T, int N>
struct Vec {
    using W = typename Word<N * static_cast<int>(sizeof(T))>::type;
    W w;
    __device__ __forceinline__ void get(float (&v)[N]) const {
        alignas(16) T x[N];
        *reinterpret_cast<W*>(x) = w;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = to_f32(x[i]);
    }
    __device__ __forceinline__ void set(const float (&v)[N]) {
        alignas(16) T x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = from_f32<T>(v[i]);
        w = *reinterpret_cast<const W*>(x);
    }
};

__device__ __forceinline__ int slot_of(const RowsParams& p, long long i) {
    const int s = __ldg(p.slots + i);
    return s >= 0 && s < p.R ? s : -1;
}

// The row from which on p.out is zeroed: a slot from there on names no row of it (whoever came last would decide what it holds).
__device__ __forceinline__ int used_rows(const RowsParams& p) { return min(max(__ldg(p.used), 0), p.R); }

// Zeros to the rows from `used` on, `worker` of `workers` threads.
template <typename T, int N>
__device__ __forceinline__ void zero_unused(const RowsParams& p, int used, long long worker, long long workers, int nvec) {
    const long long n = static_cast<long long>(p.R - used) * nvec;
    for (long long i = worker; i < n; i += workers) {
        const long long r = i / nvec;
        const int c = static_cast<int>(i - r * nvec) * N;
        T* o = static_cast<T*>(p.out) + (used + r) * p.ldo + c;
        if (c + N <= p.H) {
            *reinterpret_cast<typename Vec<T, N>::W*>(o) = typename Vec<T, N>::W{};
        } else {
            for (int j = 0; c + j < p.H; ++j) o[j] = from_f32<T>(0.f);
        }
    }
}

// A vector of a row, `left` elements before the row's end; zeros past it.
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T* p, int left) {
    using W = typename Vec<T, N>::W;
    Vec<T, N> x;
    if (left >= N) {
        x.w = __ldg(reinterpret_cast<const W*>(p));
    } else {
        alignas(16) T e[N];
#pragma unroll
        for (int j = 0; j < N; ++j) e[j] = j < left ? p[j] : from_f32<T>(0.f);
        x.w = *reinterpret_cast<const W*>(e);
    }
    return x;
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, N>& x, int left) {
    using W = typename Vec<T, N>::W;
    if (left >= N) {
        *reinterpret_cast<W*>(p) = x.w;
    } else {
        alignas(16) T e[N];
        *reinterpret_cast<W*>(e) = x.w;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < left) p[j] = e[j];
    }
}

// Which token and which of its `per` threads a thread is.
__device__ __forceinline__ bool token_of(const RowsParams& p, uint32_t per, uint32_t& t, uint32_t& v) {
    const uint32_t id = blockIdx.x * kRowsThreads + threadIdx.x;
    t = id / per;
    v = id - t * per;
    return t < static_cast<uint32_t>(p.T);
}

// A thread: U vectors of a token's row, `per` vectors apart.
template <typename T, int N, int U>
__global__ void __launch_bounds__(kRowsThreads) spread_kernel(const RowsParams p, uint32_t nvec, uint32_t per) {
    const int used = used_rows(p);
    uint32_t t, v;
    if (token_of(p, per, t, v)) {
        const T* x = static_cast<const T*>(p.X) + t * p.ldx;
        Vec<T, N> row[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u * per < nvec) row[u] = load_vec<T, N>(x + (v + u * per) * N, p.H - (v + u * per) * N);
        const long long first = static_cast<long long>(t) * p.k;
        for (int j = 0; j < p.k; ++j) {
            const int s = slot_of(p, first + j);
            if (s < 0 || s >= used) continue;
            T* y = static_cast<T*>(p.out) + s * p.ldo;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v + u * per < nvec) store_vec<T, N>(y + (v + u * per) * N, row[u], p.H - (v + u * per) * N);
        }
    }
    if (p.zero)
        zero_unused<T, N>(p, used, blockIdx.x * static_cast<long long>(kRowsThreads) + threadIdx.x,
                          static_cast<long long>(gridDim.x) * kRowsThreads, nvec);
}

// A thread: U vectors of a token's result, B choices at a time; all loads of a
// batch are under way before the first is used.
template <typename T, int N, int B, int U>
__global__ void __launch_bounds__(kRowsThreads) combine_kernel(const RowsParams p, uint32_t nvec, uint32_t per) {
    uint32_t t, v;
    if (!token_of(p, per, t, v)) return;
    const long long first = static_cast<long long>(t) * p.k;
    float sum[U][N] = {};
    for (int j0 = 0; j0 < p.k; j0 += B) {
        Vec<T, N> y[B][U];
        int slot[B];
        float w[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            slot[b] = j0 + b < p.k ? slot_of(p, first + j0 + b) : -1;
            w[b] = slot[b] >= 0 && p.weights ? __ldg(p.weights + first + j0 + b) : 1.f;
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const T* row = static_cast<const T*>(p.Y) + slot[b] * p.ldy;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (slot[b] >= 0 && v + u * per < nvec)
                    y[b][u] = load_vec<T, N>(row + (v + u * per) * N, p.H - (v + u * per) * N);
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (slot[b] >= 0) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float x[N];
                    y[b][u].get(x);
#pragma unroll
                    for (int i = 0; i < N; ++i) sum[u][i] = fmaf(w[b], x[i], sum[u][i]);
                }
            }
    }
    T* o = static_cast<T*>(p.out) + t * p.ldo;
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (v + u * per < nvec) {
            Vec<T, N> x;
            x.set(sum[u]);
            store_vec<T, N>(o + (v + u * per) * N, x, p.H - (v + u * per) * N);
        }
}

// A token to `group` threads (a power of two, 32 to 256), B choices at a time, U
// vectors a thread and round.
template <typename T, int N, int B, int U>
__global__ void __launch_bounds__(kRowsThreads) combine_grad_kernel(const RowsParams p, int nvec, int group) {
    __shared__ float part[kRowsThreads / 32][B];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int member = threadIdx.x & (group - 1);
    const uint32_t t = blockIdx.x * (kRowsThreads / group) + threadIdx.x / group;
    const bool there = t < static_cast<uint32_t>(p.T);
    const T* const dx = static_cast<const T*>(p.X) + t * p.ldx;
    const long long first = static_cast<long long>(t) * p.k;
    const int used = p.out ? used_rows(p) : 0;
    for (int j0 = 0; j0 < p.k; j0 += B) {
        int slot[B];
        float w[B], dot[B] = {};
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const bool in = there && j0 + b < p.k;
            slot[b] = in ? slot_of(p, first + j0 + b) : -1;
            w[b] = in && p.weights ? __ldg(p.weights + first + j0 + b) : 1.f;
        }
        for (int v = member; there && v < nvec; v += U * group) {
            Vec<T, N> d[U], y[B][U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v + u * group < nvec) d[u] = load_vec<T, N>(dx + (v + u * group) * N, p.H - (v + u * group) * N);
            if (p.dweights) {  // (all loads before the first use)
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const T* row = static_cast<const T*>(p.Y) + slot[b] * p.ldy;
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (slot[b] >= 0 && v + u * group < nvec)
                            y[b][u] = load_vec<T, N>(row + (v + u * group) * N, p.H - (v + u * group) * N);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (v + u * group >= nvec) continue;
                float x[N];
                d[u].get(x);
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    if (slot[b] < 0) continue;
                    float z[N];
                    if (p.dweights) {
                        y[b][u].get(z);
#pragma unroll
                        for (int i = 0; i < N; ++i) dot[b] = fmaf(x[i], z[i], dot[b]);
                    }
                    if (slot[b] < used) {
                        Vec<T, N> o;
#pragma unroll
                        for (int i = 0; i < N; ++i) z[i] = w[b] * x[i];
                        o.set(z);
                        store_vec<T, N>(static_cast<T*>(p.out) + slot[b] * p.ldo + (v + u * group) * N, o,
                                        p.H - (v + u * group) * N);
                    }
                }
            }
        }
        if (p.dweights) {
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
                for (int s = 16; s; s /= 2) dot[b] += __shfl_xor_sync(kAll, dot[b], s);
            if (group > 32) {
                if (lane == 0) {
#pragma unroll
                    for (int b = 0; b < B; ++b) part[warp][b] = dot[b];
                }
                __syncthreads();
                if (member < B && there && j0 + member < p.k) {
                    float sum = 0.f;
                    for (int q = 0; q < group / 32; ++q) sum += part[warp + q][member];
                    p.dweights[first + j0 + member] = sum;
                }
                __syncthreads();
            } else if (there) {
#pragma unroll
                for (int b = 0; b < B; ++b)
                    if (lane == b && j0 + b < p.k) p.dweights[first + j0 + b] = dot[b];
            }
        }
    }
    if (p.zero)
        zero_unused<T, N>(p, used, blockIdx.x * static_cast<long long>(kRowsThreads) + threadIdx.x,
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

// f(integral_constant<B>, integral_constant<U>): choices at a time and vectors
// of each, up to 8 loads in flight a thread.  Measured, us (floor 45 / 84; 49 / 89;
// 69 / 104), a combination / its gradient of 8192 tokens and 8 choices of 2048 bf16:
// (8, 1) 54 / 112, (4, 2) 49 / 94, (4, 1) 49 / 93; 8192 tokens, 4 choices of 4096:
// (4, 2) 56 / 99, (2, 4) 54 / 99, one load at a time 99 / 165; 16384 tokens, one choice of
// 7168: (1, 4) 87 / 103, (1, 8) 85 / 112, one load 128 / 332.  64 tokens, 4 choices of
// 4096: (4, 2) 2.2 / 3.5, (2, 4) 2.4 / 5.4.
template <typename F>
int by_choices(int k, F f) {
    if (k > 2) return f(std::integral_constant<int, 4>(), std::integral_constant<int, 2>());
    if (k > 1) return f(std::integral_constant<int, 2>(), std::integral_constant<int, 4>());
    return f(std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
}

// Launches for tokens in parts that a 32-bit thread number holds: launch(part,
// threads) with the arrays' beginnings moved to each part's.
template <typename L>
int in_parts(const RowsParams& p, int size, long long per, L launch) {
    const int most = static_cast<int>(std::max(1ll, (1ll << 30) / per));  // (per >= 1: an int holds it)
    int t0 = 0;
    do {
        RowsParams q = p;
        q.T = std::min(most, p.T - t0);
        const long long at = t0, row = at * p.k;
        if (p.X) q.X = static_cast<const char*>(p.X) + at * p.ldx * size;
        q.slots = p.slots + row;
        if (p.weights) q.weights = p.weights + row;
        if (p.dweights) q.dweights = p.dweights + row;
        if (!p.X && p.out) q.out = static_cast<char*>(p.out) + at * p.ldo * size;  // (a combination's result goes by token)
        q.zero = p.used && t0 == 0;
        const int rc = launch(q, q.T * per);
        if (rc != SGEMM_OK) return rc;
        t0 += q.T;
    } while (t0 < p.T);
    return SGEMM_OK;
}

unsigned ctas_for(long long threads, int least) {
    return static_cast<unsigned>(std::max<long long>((threads + kRowsThreads - 1) / kRowsThreads, least));
}

int launched() { return cudaGetLastError() == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA; }

}  // namespace

int rows_spread(const RowsParams& p, int type, int sms, cudaStream_t s) {
    const uint32_t nvec = static_cast<uint32_t>((p.H + p.vec - 1) / p.vec);
    return by_type_and_vec(type, p.vec, [&](auto zero, auto vec) {
        // (two vectors a thread where there are threads enough)
        const bool two = static_cast<long long>(p.T) * nvec >= 4096ll * sms;
        const uint32_t per = two ? (nvec + 1) / 2 : nvec;
        return in_parts(p, sizeof(zero), per, [&](const RowsParams& q, long long threads) {
            const unsigned ctas = ctas_for(threads, q.zero ? sms : 1);  // (the rows to zero are shared among all)
            if (two)
                spread_kernel<decltype(zero), decltype(vec)::value, 2><<<ctas, kRowsThreads, 0, s>>>(q, nvec, per);
            else
                spread_kernel<decltype(zero), decltype(vec)::value, 1><<<ctas, kRowsThreads, 0, s>>>(q, nvec, per);
            return launched();
        });
    });
}

int rows_combine(const RowsParams& p, int type, int sms, cudaStream_t s) {
    const uint32_t nvec = static_cast<uint32_t>((p.H + p.vec - 1) / p.vec);
    return by_type_and_vec(type, p.vec, [&](auto zero, auto vec) {
        return by_choices(p.k, [&](auto b, auto u) {
            using T = decltype(zero);
            constexpr int N = decltype(vec)::value, B = decltype(b)::value, U = decltype(u)::value;
            const bool wide = U > 1 && static_cast<long long>(p.T) * nvec >= 2048ll * U * sms;
            const uint32_t per = wide ? (nvec + U - 1) / U : nvec;
            return in_parts(p, sizeof(T), per, [&](const RowsParams& q, long long threads) {
                if (wide)
                    combine_kernel<T, N, B, U><<<ctas_for(threads, 1), kRowsThreads, 0, s>>>(q, nvec, per);
                else
                    combine_kernel<T, N, B, 1><<<ctas_for(threads, 1), kRowsThreads, 0, s>>>(q, nvec, per);
                return launched();
            });
        });
    });
}

int rows_combine_grad(const RowsParams& p, int type, int sms, cudaStream_t s) {
    const int nvec = (p.H + p.vec - 1) / p.vec;
    return by_type_and_vec(type, p.vec, [&](auto zero, auto vec) {
        return by_choices(p.k, [&](auto b, auto u) {
            using T = decltype(zero);
            constexpr int N = decltype(vec)::value, B = decltype(b)::value, U = decltype(u)::value;
            // Threads a token: two rounds of vectors each; more where there are few tokens.
            int group = 32;
            while (group < kRowsThreads && (nvec > 2 * U * group || (nvec > U * group && static_cast<long long>(p.T) * group < 1024ll * sms)))
                group *= 2;
            return in_parts(p, sizeof(T), group, [&](const RowsParams& q, long long threads) {
                combine_grad_kernel<T, N, B, U><<<ctas_for(threads, q.zero ? sms : 1), kRowsThreads, 0, s>>>(q, nvec, group);
                return launched();
            });
        });
    });
}

}  // namespace gb300
