// Grouped float32 products of few rows an expert, on the CUDA cores.
//
// With a few rows an expert the product costs what reading the
// weights costs, once, 4 bytes each; the tensor-core path would write three
// bf16 parts of them first (10 bytes more, and 6 read).  So here a weight goes
// from HBM to a register and meets RT rows of its group, whose values lie in
// shared memory; longer groups take ceil(rows / RT) tiles.  float32 products
// and sums throughout.
//
// A CTA of 8 warps computes RT rows x kCols columns over its part of the
// contraction, in chunks of 512 whose X values all threads copy to shared memory:
//   plain (W stored K x N): kCols = 128, four columns a lane; the warps take
//     every eighth k, and their sums meet in shared memory in the warps' order;
//   transposed (N x K): kCols = 32, four columns a warp, four k a lane; the
//     lanes' sums meet by shuffles.
// Where tiles are few, the contraction is split over a cluster of up to 8 CTAs
// that add their parts in rank order through each other's shared memory.
// Measured for 32 / 64 rows, 8 experts of 1024 x 2048 (67 MB of weights): 13 / 19
// us (5.0 / 3.6 TB/s), transposed 14 / 21; 50 by parts.  Up to 4 rows a group it
// is the weights' bytes that bound it, from 8 on the multiply-adds' issue.
#include "../../include/sgemm_experts.h"
#include "api_internal.h"
#include "experts.h"
#include "experts_groups.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace detail {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kChunk = 512;
// Contraction after which a thread's sums are put by: 512 additions in a row at
// most stay below 512 * 2^-24 = 3.1e-5 of the sum of magnitudes, whatever the
// operands.  Kernels of their own (LONG) do so: the loop around the chunks alone
// costs the transposed form a fifth (32 rows, 8 experts of 1024 x 2048 17 -> 21 us).
template <bool TRANS>
constexpr int kInARow = (TRANS ? 32 : 8) * kChunk;

struct FewParams {
    const float* X;
    const float* W;
    float* Y;
    long long ldx, ldw, sw, ldy;
    const int* offsets;
    int T, E, N, K;
    int ks;  // CTAs a tile's contraction is split over
    int per; // and the contraction of each
};

template <bool TRANS>
constexpr int kCols = TRANS ? 32 : 128;

// X's values, and for the plain form the warps' sums.
template <bool TRANS, int RT>
constexpr int kSmemFloats = RT * kChunk + (TRANS ? 0 : kWarps * RT * 128);

__device__ __forceinline__ float4 load4(const float* p, int n, bool vec) {
    if (vec && n >= 4) return __ldg(reinterpret_cast<const float4*>(p));
    return make_float4(n > 0 ? __ldg(p) : 0.f, n > 1 ? __ldg(p + 1) : 0.f, n > 2 ? __ldg(p + 2) : 0.f,
                       n > 3 ? __ldg(p + 3) : 0.f);
}

template <bool TRANS, int RT, bool LONG>
__global__ void __launch_bounds__(kThreads) few_kernel(const FewParams p) {
    extern __shared__ float sm[];
    __shared__ GroupHit hit;
    __shared__ int found;
    __shared__ float part[RT * kCols<TRANS>];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = p.ks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int c0 = static_cast<int>(blockIdx.x) / p.ks * kCols<TRANS>;
    if (warp == 0) {
        GroupCursor cur = group_begin(p.offsets, p.T);
        GroupHit h;
        const bool ok =
            group_find(p.offsets, p.E, p.T, blockIdx.y, cur, [](int n) { return (n + RT - 1) / RT; }, h);
        if (lane == 0) {
            hit = h;
            found = ok;
        }
    }
    __syncthreads();
    if (found) {  // (all CTAs of a cluster alike)
        const int r0 = hit.start + hit.local * RT, rows = min(RT, hit.end - r0);
        const float* const W = p.W + hit.e * p.sw;
        const int kbeg = min(p.K, rank * p.per), kend = min(p.K, kbeg + p.per);
        float acc[RT][4] = {};
        float* const sums = sm + RT * kChunk + (warp * RT * 128 + 4 * lane);  // (plain form: 128 apart)
        // The sums in `acc` to shared memory: the thread's own, or (transposed) over the lanes, one of which owns each.
        auto put_by = [&](bool first) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if constexpr (!TRANS) {
                    float4* const at = reinterpret_cast<float4*>(sums + r * 128);
                    float4 v = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
                    if (!first) v = make_float4(at->x + v.x, at->y + v.y, at->z + v.z, at->w + v.w);
                    *at = v;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (TRANS) {
                        float s = acc[r][j];
#pragma unroll
                        for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
                        float* const at = part + r * 32 + 4 * warp + j;
                        if (lane == (r * 4 + j) % 32) *at = first ? s : *at + s;
                    }
                    acc[r][j] = 0.f;
                }
            }
        };
        int from = kbeg;
        do {
            const int to = LONG ? min(kend, from + kInARow<TRANS>) : kend;
            for (int k0 = from; k0 < to; k0 += kChunk) {
                const int len = min(kChunk, kend - k0);
                __syncthreads();
                // X's values: [k][row] for the plain form, [row][k] for the other; zeros past the rows and the end.
                for (int i = threadIdx.x; i < RT * kChunk; i += kThreads) {
                    const int r = i / kChunk, k = i % kChunk;
                    const float v = r < rows && k < len ? __ldg(p.X + (r0 + r) * p.ldx + k0 + k) : 0.f;
                    sm[TRANS ? i : k * RT + r] = v;
                }
                __syncthreads();
                if constexpr (!TRANS) {
                    const int c = c0 + 4 * lane, n = p.N - c;
                    const float* w0 = W + static_cast<long long>(k0) * p.ldw + c;
                    const bool vec = (reinterpret_cast<uintptr_t>(w0) & 15) == 0 && p.ldw % 4 == 0;
                    constexpr int kU = 8;  // loads under way
                    static_assert(kChunk % (kWarps * kU) == 0, "steps do not pass the chunk");
                    for (int k = warp; k < len; k += kWarps * kU) {
                        float4 w[kU];
#pragma unroll
                        for (int u = 0; u < kU; ++u) {
                            const int kk = k + u * kWarps;
                            w[u] = load4(w0 + kk * p.ldw, kk < len ? n : 0, vec);
                        }
#pragma unroll
                        for (int u = 0; u < kU; ++u) {
                            // (inside the chunk: k < kChunk - (kU - 1) kWarps; past its end both are 0)
                            const float4* x = reinterpret_cast<const float4*>(sm + (k + u * kWarps) * RT);
#pragma unroll
                            for (int r = 0; r < RT; r += 4) {
                                const float4 v = x[r / 4];
                                const float xs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    acc[r + i][0] = fmaf(xs[i], w[u].x, acc[r + i][0]);
                                    acc[r + i][1] = fmaf(xs[i], w[u].y, acc[r + i][1]);
                                    acc[r + i][2] = fmaf(xs[i], w[u].z, acc[r + i][2]);
                                    acc[r + i][3] = fmaf(xs[i], w[u].w, acc[r + i][3]);
                                }
                            }
                        }
                    }
                } else {
                    const int c = c0 + 4 * warp;
                    const bool vec = p.ldw % 4 == 0 && (reinterpret_cast<uintptr_t>(W + k0) & 15) == 0;
                    for (int k = 4 * lane; k < len; k += 256) {  // two steps of 128 k under way
                        float4 w[2][4];
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int kk = k + 128 * u;
                                w[u][j] = load4(W + (c + j) * p.ldw + k0 + kk, c + j < p.N ? len - kk : 0, vec);
                            }
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int kk = k + 128 * u;  // (k < kChunk - 128: inside the chunk; past its end both are 0)
#pragma unroll
                            for (int r = 0; r < RT; ++r) {
                                const float4 x = *reinterpret_cast<const float4*>(sm + r * kChunk + kk);
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    acc[r][j] = fmaf(x.x, w[u][j].x, acc[r][j]);
                                    acc[r][j] = fmaf(x.y, w[u][j].y, acc[r][j]);
                                    acc[r][j] = fmaf(x.z, w[u][j].z, acc[r][j]);
                                    acc[r][j] = fmaf(x.w, w[u][j].w, acc[r][j]);
                                }
                            }
                        }
                    }
                }
            }
            put_by(!LONG || from == kbeg);
            from = to;
        } while (LONG && from < kend);
        // The CTA's sums, to `part`.
        __syncthreads();
        if constexpr (!TRANS) {
            for (int i = threadIdx.x; i < RT * 128; i += kThreads) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += sm[RT * kChunk + w * RT * 128 + i];
                part[i] = s;
            }
        }
        __syncthreads();
        if (p.ks > 1) cluster_sync_all();  // the others' parts are there
        // Rows of the tile in turn to the cluster's CTAs.
        const uint32_t mine = smem_addr(part);
        for (int i = threadIdx.x; i < RT * kCols<TRANS>; i += kThreads) {
            const int r = i / kCols<TRANS>, c = c0 + i % kCols<TRANS>;
            if (r % p.ks != rank || r >= rows || c >= p.N) continue;
            float s = 0.f;
            if (p.ks == 1) {
                s = part[i];
            } else {
                for (int q = 0; q < p.ks; ++q) s += ld_shared_cluster_f32(map_shared_rank(mine + 4 * i, q));
            }
            p.Y[(r0 + r) * p.ldy + c] = s;
        }
        if (p.ks > 1) cluster_sync_all();  // nobody's part is still being read
    }
    // Rows of no expert: zeros, by the first row of CTAs.
    if (blockIdx.y == 0 && rank == 0) {
        const int first = group_bound(p.offsets, 0, p.T);
        int last = first;
        for (int i = lane; i <= p.E; i += 32) last = max(last, group_bound(p.offsets, i, p.T));
        last = __reduce_max_sync(0xffffffffu, last);
        const int none = first + p.T - last;
        for (int i = threadIdx.x; i < kCols<TRANS>; i += kThreads)
            if (c0 + i < p.N)
                for (int r = 0; r < none; ++r)
                    p.Y[static_cast<long long>(r < first ? r : last + r - first) * p.ldy + c0 + i] = 0.f;
    }
}

template <bool TRANS, int RT>
int launch(FewParams p, int sms, cudaStream_t s) {
    const long long cols = ceil_div(p.N, kCols<TRANS>), tiles = p.T / RT + std::min(p.T, p.E);
    // Split the contraction while that leaves a CTA an SM at most (a CTA reads 64 k at a time and waits: 39 rows, 8
    // experts of 896 x 192 21 us on 16 CTAs of 896 k, 11 on 64), in parts of 128 or more.  (Two CTAs an SM: 17 us
    // instead of 12 for 32 rows, 8 experts of 1024 x 2048.)
    p.ks = 1;
    while (p.ks < 8 && 2 * p.ks * cols * std::min(p.T, p.E) <= sms && p.K >= 2 * p.ks * 128) p.ks *= 2;
    p.per = ((p.K + p.ks - 1) / p.ks + 127) & ~127;  // (parts begin on vectors)
    if (tiles > 65535 || cols * p.ks > 0x7fffffffll) return SGEMM_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cols * p.ks), static_cast<unsigned>(tiles));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemFloats<TRANS, RT> * sizeof(float);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(p.ks);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = p.ks > 1 ? 1 : 0;
    const auto kernel = p.per > kInARow<TRANS> ? few_kernel<TRANS, RT, true> : few_kernel<TRANS, RT, false>;
    if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

template <bool TRANS, int RT>
int set_up() {
    for (const auto kernel : {few_kernel<TRANS, RT, false>, few_kernel<TRANS, RT, true>})
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmemFloats<TRANS, RT> * sizeof(float)) != cudaSuccess)
            return SGEMM_ERR_CUDA;
    return SGEMM_OK;
}

}  // namespace

int experts_few_set_up() {
    if (set_up<false, 4>() || set_up<false, 8>() || set_up<true, 4>() || set_up<true, 8>()) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

int grouped_few(const GroupedCall& c, const DeviceState& st, cudaStream_t s) {
    FewParams p = {};
    p.X = static_cast<const float*>(c.b.p), p.W = static_cast<const float*>(c.a.p), p.Y = static_cast<float*>(c.out);
    p.ldx = c.b.ld, p.ldw = c.a.ld, p.sw = c.a.se, p.ldy = c.ldo;
    p.offsets = c.offsets;
    p.T = c.T, p.E = c.E, p.N = c.F, p.K = c.K;
    // (4 rows a tile where groups have no more on average: a quarter of the multiply-adds)
    const bool four = c.T <= 4ll * std::min(c.T, c.E);
    if (c.a_mn) return four ? launch<false, 4>(p, st.sm_count, s) : launch<false, 8>(p, st.sm_count, s);
    return four ? launch<true, 4>(p, st.sm_count, s) : launch<true, 8>(p, st.sm_count, s);
}

}  // namespace detail
}  // namespace gb300
