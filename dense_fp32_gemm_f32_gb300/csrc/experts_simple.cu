// Grouped products on the CUDA cores: one 64 x 64 tile of the output per CTA,
// slices of 16 along the contraction through shared memory, 4 x 4 float32
// accumulators a thread.  Any type, stride and alignment.
#include "../../include/sgemm_experts.h"
#include "experts.h"
#include "experts_groups.cuh"

namespace gb300 {
namespace {

constexpr int kT = 64, kS = 16;

template <typename T>
struct StridedLoad {
    StridedOperand o;
    __device__ float operator()(int e, long long r, long long k, long long) const {
        return to_f32(static_cast<const T*>(o.p)[e * o.se + r * o.sr + k * o.sk]);
    }
};

__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const float m[8] = {0.f, .5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
    const float v = m[c & 7];
    return c & 8 ? -v : v;
}

// `sr`: the row's place among the scale blocks' rows.
struct Mxfp4Load {
    Mxfp4Operand o;
    __device__ float operator()(int e, long long r, long long k, long long sr) const {
        const uint8_t b = o.codes[e * o.codes_e + r * o.pitch + (k >> 1)];
        const long long blk = k >> 5;
        const uint8_t s =
            o.scales[e * o.scales_e + ((sr >> 7) * o.kq + (blk >> 2)) * 512 + (sr & 31) * 16 + ((sr & 127) >> 5) * 4 +
                     (blk & 3)];
        const float scale = s == 255 ? __int_as_float(0x7fffffff)
                                     : __int_as_float(s == 0 ? 0x00400000 : static_cast<int>(s) << 23);
        return e2m1_value(k & 1 ? b >> 4 : b & 15) * scale;
    }
};

// One tile: sum over k of a(r, k) b(c, k), r < nr, c < nc.
template <typename FA, typename FB>
__device__ void tile_product(float (&acc)[4][4], int nr, int nc, int K, FA a, FB b) {
    __shared__ float As[kS][kT + 1], Bs[kS][kT + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int k0 = 0; k0 < K; k0 += kS) {
        for (int i = threadIdx.x; i < kS * kT; i += 256) {
            const int r = i / kS, k = i % kS;
            As[k][r] = r < nr && k0 + k < K ? a(r, k0 + k) : 0.f;
            Bs[k][r] = r < nc && k0 + k < K ? b(r, k0 + k) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kS; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(As[k][ty * 4 + i], Bs[k][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
}

template <typename TO>
__device__ void store_tile(const float (&acc)[4][4], TO* out, long long ld, int nr, int nc) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
            if (ty * 4 + i < nr && tx * 4 + j < nc) out[(ty * 4 + i) * ld + tx * 4 + j] = from_f32<TO>(acc[i][j]);
}

template <typename LA, typename LB, typename TO>
__global__ void __launch_bounds__(256) forward_kernel(LA la, LB lb, const SimpleParams p) {
    __shared__ GroupHit sh;
    __shared__ int found;
    TO* const out = static_cast<TO*>(p.out);
    const int c0 = blockIdx.x * kT, nc = min(kT, p.N - c0);
    if (!p.offsets) {
        if (threadIdx.x == 0) {
            sh = {0, 0, p.T, static_cast<int>(blockIdx.y), 0};
            found = static_cast<int>(blockIdx.y) * kT < p.T;
        }
    } else if (threadIdx.x < 32) {
        GroupCursor cur = group_begin(p.offsets, p.T);
        GroupHit h;
        const bool ok = group_find(
            p.offsets, p.E, p.T, blockIdx.y, cur, [](int n) { return (n + kT - 1) / kT; }, h);
        if (threadIdx.x == 0) {
            sh = h;
            found = ok;
        }
    }
    __syncthreads();
    if (found) {
        const int r0 = sh.start + sh.local * kT, nr = min(kT, sh.end - r0), e = sh.e;
        const long long s0 = 128ll * sh.block0 + sh.local * kT;
        float acc[4][4] = {};
        tile_product(
            acc, nr, nc, p.K, [&](int r, int k) { return la(0, r0 + r, k, s0 + r); },
            [&](int c, int k) { return lb(e, c0 + c, k, c0 + c); });
        store_tile(acc, out + static_cast<long long>(r0) * p.ldo + c0, p.ldo, nr, nc);
    }
    if (p.offsets && blockIdx.y == gridDim.y - 1) {  // rows of no expert
        const int first = group_bound(p.offsets, 0, p.T);
        int last = first;
        for (int i = 1; i <= p.E; ++i) last = max(last, group_bound(p.offsets, i, p.T));
        for (long long t = 0; t < p.T; ++t) {
            if (t == first) t = last;
            if (t < p.T && threadIdx.x < nc) out[t * p.ldo + c0 + threadIdx.x] = from_f32<TO>(0.f);
        }
    }
}

template <typename T, typename TO>
__global__ void __launch_bounds__(256) wgrad_kernel(StridedLoad<T> la, StridedLoad<T> lb, const SimpleParams p) {
    const int e = blockIdx.z;
    int start = group_bound(p.offsets, 0, p.T), end = start;
    for (int i = 0; i <= e; ++i) {
        start = end;
        end = max(end, group_bound(p.offsets, i + 1, p.T));
    }
    const int r0 = blockIdx.y * kT, c0 = blockIdx.x * kT;
    const int nr = min(kT, p.R - r0), nc = min(kT, p.N - c0);
    float acc[4][4] = {};
    tile_product(
        acc, nr, nc, end - start, [&](int r, int k) { return la(0, r0 + r, start + k, 0); },
        [&](int c, int k) { return lb(0, c0 + c, start + k, 0); });
    store_tile(acc, static_cast<TO*>(p.out) + e * p.so + r0 * p.ldo + c0, p.ldo, nr, nc);
}

int status() {
    if (cudaGetLastError() != cudaSuccess) return SGEMM_ERR_CUDA;
    return SGEMM_OK;
}

dim3 forward_grid(const SimpleParams& p) {
    return dim3((p.N + kT - 1) / kT, p.offsets ? p.T / kT + (p.E < p.T ? p.E : p.T) + 1 : (p.T + kT - 1) / kT);
}

template <int TYPE>
int forward_t(const SimpleParams& p, cudaStream_t s) {
    using T = typename ElemOf<TYPE>::T;
    forward_kernel<StridedLoad<T>, StridedLoad<T>, T>
        <<<forward_grid(p), 256, 0, s>>>(StridedLoad<T>{p.A}, StridedLoad<T>{p.B}, p);
    return status();
}

template <int TYPE>
int mxfp4_t(const SimpleParams& p, cudaStream_t s) {
    forward_kernel<Mxfp4Load, Mxfp4Load, typename ElemOf<TYPE>::T>
        <<<forward_grid(p), 256, 0, s>>>(Mxfp4Load{p.qA}, Mxfp4Load{p.qB}, p);
    return status();
}

template <int TYPE, int OTYPE>
int wgrad_t(const SimpleParams& p, cudaStream_t s) {
    using T = typename ElemOf<TYPE>::T;
    using TO = typename ElemOf<OTYPE>::T;
    wgrad_kernel<T, TO><<<dim3((p.N + kT - 1) / kT, (p.R + kT - 1) / kT, p.E), 256, 0, s>>>(
        StridedLoad<T>{p.A}, StridedLoad<T>{p.B}, p);
    return status();
}

}  // namespace

int simple_forward(const SimpleParams& p, int type, cudaStream_t s) {
    return type == 0 ? forward_t<0>(p, s) : type == 1 ? forward_t<1>(p, s) : forward_t<2>(p, s);
}

int simple_mxfp4(const SimpleParams& p, int type, cudaStream_t s) {
    return type == 0 ? mxfp4_t<0>(p, s) : type == 1 ? mxfp4_t<1>(p, s) : mxfp4_t<2>(p, s);
}

int simple_wgrad(const SimpleParams& p, int type, int out_type, cudaStream_t s) {
    if (out_type == 0) return type == 0 ? wgrad_t<0, 0>(p, s) : type == 1 ? wgrad_t<1, 0>(p, s) : wgrad_t<2, 0>(p, s);
    return type == 1 ? wgrad_t<1, 1>(p, s) : wgrad_t<2, 2>(p, s);
}

}  // namespace gb300
