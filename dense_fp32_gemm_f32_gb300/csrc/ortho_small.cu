// Orthogonalised updates of matrices with a short side of up to 128 (X: m x n, m
// <= 128): all steps in one launch that keeps X in shared memory.
//
// A cluster of CTAs takes a matrix, W columns of X a CTA.  The mathematics,
// planes and scales are those of ortho_tc.cuh.  X lies in shared memory as 64
// columns of 128 rows a block, rows of 128 bytes (128-byte swizzle), which the
// tensor core reads as either operand of X X^T (the columns are the contraction:
// K-major) and as the second of B X (rows the contraction: MN-major).  So a step
// is three products without a copy in between, each waited for:
//
//   gram     a CTA's part of A = X X^T.  With several CTAs the parts are summed
//            through distributed shared memory, each CTA some of the rows, in the
//            CTAs' order, and sent to all
//   square   B = b A + c A A, in every CTA
//   update   X = a X + B X, a CTA's own columns
//
// A thread has a row (its lane of tensor memory) and a quarter of the columns, and what
// it reads and writes of a plane between products are its own elements, so that
// each plane is updated in place.
//
// Bound by latency: five steps of three dependent products, each a barrier, 6 to 16
// instructions of the tensor core for each product of planes, and about 450 instructions a
// warp to put its sums back (a quarter of the issue slots are used).  Measured on GB300, five steps, products of
// one plane and of two: 64 x 64 24 and 29 us, 128 x 96 31 and 40 us, 128 x 512 56 and 67 us (4 CTAs; the sums
// of their parts 3 us a step).  (What follows was measured with one plane for bf16, two for float32.)  Of 128 x 96 40 and 48 us before what a thread updates was loaded while the product
// runs, G read once and a row of the diagonal four values a load.  The many-tile form
// (ortho_tc.cuh) took 71 and 102 us, most of it on the way of tiles through HBM;
// 8 warps, half as many as here, 49 and 57 when these were 41 and 49.
#include "../../include/sgemm_ortho.h"
#include "api_internal.h"
#include "experts_tc.cuh"
#include "ortho.h"
#include "ortho_load.cuh"

namespace gb300 {
namespace detail {
namespace {

constexpr int kSmallThreads = 512, kSmallShare = kSmallThreads / 128;  // warps that share a quarter of the rows
constexpr int kSmallBlock = 128 * 128;  // bytes of 64 columns of a plane (or of 64 of A's)

struct OrthoSmallParams {
    const void* G;
    long long ldg, sg;
    void* out;
    long long ldo, so;
    int m, n, steps, width;  // width: CTAs of a cluster
    int vec, align;          // G's rows begin on 16 bytes; bytes that the result's are aligned to
    float c1, c3, c5;
    int growth;
    double eps;
    unsigned long long timeout_ns;
    unsigned int* status;
};

template <int W, int PARTS>
struct SmallShape {
    static constexpr int kXBytes = W / 64 * kSmallBlock, kABytes = 2 * kSmallBlock;  // of a plane
    static constexpr int kPlanes = 2 * kXBytes + 2 * kABytes;
    static constexpr int kTmemCols = PARTS * W;
    // d, e: 128 floats each; the CTAs' sums and scratch: 16 + 16 doubles; a barrier; the address of tensor memory
    static constexpr int kSmem = kPlanes + 2 * 512 + (16 + kSmallThreads / 32) * 8 + 16 + 1024;
    static_assert(kSmem <= 227 * 1024 && kTmemCols <= 512 && (W == 128 || W == 256), "shape");
};

// Byte of the 16-byte piece of columns c .. c + 7 (c a multiple of 8) of a plane's row.
__device__ __forceinline__ uint32_t piece(int row, int c) {
    return static_cast<uint32_t>((c >> 6) * kSmallBlock + row * 128 + (((c >> 3) ^ row) & 7) * 16);
}

__device__ __forceinline__ uint4 lds_u4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts_u4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float lds_f(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts_f(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_b64(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ void unpack2(uint32_t h, uint32_t l, float& a, float& b) {
    const __half2 x = *reinterpret_cast<const __half2*>(&h), y = *reinterpret_cast<const __half2*>(&l);
    a = __low2float(x) + __low2float(y);
    b = __high2float(x) + __high2float(y);
}
// Two values as f16 and what that leaves.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(a, b);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = pair_from_f32<__half>(a - __low2float(h), b - __high2float(h));
}

// 32 values of a row, columns c .., from or to its two planes.
__device__ __forceinline__ void load_planes(uint32_t hi, uint32_t lo, int row, int c, float (&x)[32]) {
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
        const uint4 h = lds_u4(hi + piece(row, c + j)), l = lds_u4(lo + piece(row, c + j));
        unpack2(h.x, l.x, x[j], x[j + 1]);
        unpack2(h.y, l.y, x[j + 2], x[j + 3]);
        unpack2(h.z, l.z, x[j + 4], x[j + 5]);
        unpack2(h.w, l.w, x[j + 6], x[j + 7]);
    }
}
__device__ __forceinline__ void store_planes(uint32_t hi, uint32_t lo, int row, int c, const float (&x)[32]) {
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
        uint4 h, l;
        split2(x[j], x[j + 1], h.x, l.x);
        split2(x[j + 2], x[j + 3], h.y, l.y);
        split2(x[j + 4], x[j + 5], h.z, l.z);
        split2(x[j + 6], x[j + 7], h.w, l.w);
        sts_u4(hi + piece(row, c + j), h);
        sts_u4(lo + piece(row, c + j), l);
    }
}

template <typename T, int W, int PARTS, bool TALL>
__global__ void __launch_bounds__(kSmallThreads, 1) ortho_small_kernel(const OrthoSmallParams p) {
    using S = SmallShape<W, PARTS>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t x_hi = base, x_lo = base + S::kXBytes;
    const uint32_t a_hi = base + 2 * S::kXBytes, a_lo = a_hi + S::kABytes;  // A's, then B's; with several CTAs first A's part
    const uint32_t d_at = base + S::kPlanes, e_at = d_at + 512, sums = e_at + 512, scratch = sums + 16 * 8;
    const uint32_t bar = scratch + 8 * (kSmallThreads / 32), tmem_slot = bar + 8, shift_at = bar + 12;

    const int warp = warp_uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int rank = warp_uniform(static_cast<int>(cluster_ctarank()));
    const int e = static_cast<int>(blockIdx.x) / p.width;
    const int n0 = rank * W, cols = min(W, p.n - n0);  // the CTA's columns of X
    const int row = 32 * (warp & 3) + lane, share = warp >> 2;
    // Rows and columns of A that are computed; what lies past them in X is zeros.  Warps of rows past them have no part.
    const int side = (p.m + 31) & ~31;
    const bool active = 32 * (warp & 3) < side;
    bool timed_out = false;

    if (threadIdx.x == 0) {
        mbar_init(bar, 1);
        fence_mbarrier_init();
    }
    __syncwarp();
    if (warp == 0) tmem_alloc_cg<1>(tmem_slot, S::kTmemCols);

    // ---------------------------------------------------------------- norm
    // The slice as it is stored: rows of X, or of X^T.
    const T* const G = static_cast<const T*>(p.G) + e * p.sg + (TALL ? n0 * p.ldg : n0);
    // A thread's octs of X: rows and columns of X, zeros where there are none.  They stay in registers until the norm is known.
    constexpr int kMine = 128 * (W / 8) / kSmallThreads;
    float g[kMine][8];
    // (neighbouring threads read neighbouring elements)
    auto row_of = [&](int u) { return TALL ? (threadIdx.x + u * kSmallThreads) & 127 : (threadIdx.x + u * kSmallThreads) / (W / 8); };
    auto column_of = [&](int u) {
        return static_cast<int>(TALL ? (threadIdx.x + u * kSmallThreads) >> 7 : (threadIdx.x + u * kSmallThreads) % (W / 8)) * 8;
    };
    if (!TALL && p.vec && cols % 8 == 0) {  // (every oct is a vector: all loads under way at once)
        alignas(16) T x[kMine][8];
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            const uint4* from = reinterpret_cast<const uint4*>(G + min(static_cast<int>(row_of(u)), p.m - 1) * p.ldg + min(column_of(u), cols - 8));
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(x[u])[i] = __ldg(from + i);
        }
#pragma unroll
        for (int u = 0; u < kMine; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) g[u][j] = row_of(u) < p.m && column_of(u) < cols ? to_f32(x[u][j]) : 0.f;
    } else {
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            const int r = row_of(u), c = column_of(u);
            if constexpr (TALL) {
#pragma unroll
                for (int j = 0; j < 8; ++j) g[u][j] = r < p.m && c + j < cols ? to_f32(G[(c + j) * p.ldg + r]) : 0.f;
            } else {
                load8(G + r * p.ldg + c, r < p.m ? cols - c : 0, p.vec, g[u]);
            }
        }
    }
    double sum = squares(g);
#pragma unroll
    for (int s = 16; s; s /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    if (lane == 0) asm volatile("st.shared.f64 [%0], %1;" ::"r"(scratch + 8 * warp), "d"(sum) : "memory");
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot) : "memory");
    tmem = warp_uniform(tmem);
    sum = 0;
    for (int w = 0; w < kSmallThreads / 32; ++w) {
        double v;
        asm volatile("ld.shared.f64 %0, [%1];" : "=d"(v) : "r"(scratch + 8 * w) : "memory");
        sum += v;
    }
    if (p.width > 1) {
        if (threadIdx.x == 0) asm volatile("st.shared.f64 [%0], %1;" ::"r"(sums), "d"(sum) : "memory");
        cluster_sync_all();
        sum = 0;
        for (int q = 0; q < p.width; ++q) sum += ld_cluster_f64(map_shared_rank(sums, q));
    }
    const double norm = sqrt(sum);
    const int shift = ortho_shift(norm, p.eps);
    // (in shared memory: between products registers are short)
    if (threadIdx.x == 0) asm volatile("st.shared.b32 [%0], %1;" ::"r"(shift_at), "r"(shift) : "memory");
    auto shift_of = [&](int step) {
        int q;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(q) : "r"(shift_at) : "memory");
        return max(0, q - step * p.growth);
    };
    const OrthoScale scale(norm + p.eps, shift);

    // ---------------------------------------------------------------- X
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
        const int r = row_of(u), c = column_of(u);
        uint4 hi = {0, 0, 0, 0}, lo = {0, 0, 0, 0};
        if (r < p.m && c < cols) scale.split(g[u], hi, lo);
        sts_u4(x_hi + piece(r, c), hi);
        sts_u4(x_lo + piece(r, c), lo);
    }

    // A product: D (128 x N) = sum over k of the first operand's rows (K-major) and the second's.  What threads
    // wrote to shared memory before is there for it, and its sums for them after.  `meanwhile`: what a warp loads
    // beside it.
    const uint64_t x_k = umma_desc_kmajor_sw128(x_hi), x_mn = umma_desc_mnmajor_sw128(x_hi, kSmallBlock);
    const uint64_t a_k = umma_desc_kmajor_sw128(a_hi);
    uint32_t phase = 0;
    auto product = [&](bool gram, bool update, int k_len, auto meanwhile) {
        fence_proxy_async_all();
        tc_fence_before_sync();
        if (p.width > 1 && !gram && !update)
            cluster_sync_all();  // (all CTAs write A)
        else
            __syncthreads();
        tc_fence_after_sync();
        if (warp == 0) {
            if (elect_one()) {
                fence_proxy_async_all();
                const int N = update ? (cols + 15) & ~15 : side;
                const uint32_t idesc = 1u << 4 | (update ? 1u << 16 : 0) | static_cast<uint32_t>(N / 8) << 17 | 8u << 24;
                for (int k = 0; k < k_len; k += 16) {
                    const uint32_t along = static_cast<uint32_t>((k >> 6) * kSmallBlock / 16 + (k & 63) / 16 * 2);
                    const uint64_t a = (gram ? x_k : a_k) + along;
                    const uint64_t b = update ? x_mn + static_cast<uint32_t>(k * 128 / 16) : a;
                    umma_f16<1>(tmem, a, b, idesc, k > 0);
                    if constexpr (PARTS == 2) {
                        const uint32_t pa = (gram ? S::kXBytes : S::kABytes) / 16, pb = (update || gram ? S::kXBytes : S::kABytes) / 16;
                        umma_f16<1>(tmem + W, a, b + pb, idesc, k > 0);
                        umma_f16<1>(tmem + W, a + pa, b, idesc, true);
                    }
                }
                umma_commit(bar);
            }
            __syncwarp();
        }
        meanwhile();
        if (!mbar_wait_warp<false>(bar, phase, p.timeout_ns)) timed_out = true;
        phase ^= 1;
        tc_fence_after_sync();
    };
    // 32 of the product's columns, from c on.
    auto sums_of = [&](int c, float (&v)[32]) {
        uint32_t r[32];
        const uint32_t at = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + static_cast<uint32_t>(c);
        __syncwarp();
        tmem_ld_32x32b_x32(at, r);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
        if constexpr (PARTS == 2) {
            tmem_ld_32x32b_x32(at + W, r);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += __uint_as_float(r[j]);
        }
    };

    static_assert(32 * kSmallShare == 128, "32 columns of A a warp");
    const int c0 = 32 * share;  // the warp's columns of A, and its first ones of X
    const bool mine = active && c0 < side;
    for (int step = 0; step < p.steps; ++step) {
        // ------------------------------------------------------------ gram
        product(true, false, cols, [] {});
        if (p.width == 1) {
            if (mine) {
                float v[32];
                sums_of(c0, v);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (c0 + j == row) {
                        sts_f(d_at + 4 * row, v[j] * 0x1p-26f);
                        v[j] = 0.f;
                    }
                    v[j] *= 0x1p-14f;
                }
                store_planes(a_hi, a_lo, row, c0, v);
            }
        } else {
            // This CTA's part, in float32: rows of 512 bytes, whose 16-byte pieces trade places by the row's number.
            auto part = [&](int r, int u) { return a_hi + static_cast<uint32_t>(r * 512 + ((u ^ r) & 31) * 16); };
            if (mine) {
                float v[32];
                sums_of(c0, v);
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    sts128(part(row, (c0 + j) / 4), make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]));
            }
            cluster_sync_all();
            // The sums of some of the rows, from all parts in their order.
            const int rows = (side + p.width - 1) / p.width, r0 = rank * rows, pieces = side / 4;
            const int items = max(0, min(rows, side - r0)) * pieces;
            constexpr int kSums = 64 * 32 / kSmallThreads;
            float4 a[kSums];
#pragma unroll
            for (int i = 0; i < kSums; ++i) {
                a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                const int item = static_cast<int>(threadIdx.x) + i * kSmallThreads;
                if (item < items) {
                    const uint32_t at = part(r0 + item / pieces, item % pieces);
#pragma unroll 4
                    for (int q = 0; q < p.width; ++q) {
                        const float4 v = ld_shared_cluster_v4(map_shared_rank(at, q));
                        a[i].x += v.x, a[i].y += v.y, a[i].z += v.z, a[i].w += v.w;
                    }
                }
            }
            cluster_sync_all();  // (all parts have been read)
#pragma unroll
            for (int i = 0; i < kSums; ++i) {
                const int item = static_cast<int>(threadIdx.x) + i * kSmallThreads;
                if (item < items) {
                    const int r = r0 + item / pieces, c = item % pieces * 4;
                    float v[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, diagonal = 0.f;
                    const bool on = r >= c && r < c + 4;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (c + j == r) {
                            diagonal = v[j] * 0x1p-26f;
                            v[j] = 0.f;
                        }
                        v[j] *= 0x1p-14f;
                    }
                    uint32_t h0, h1, l0, l1;
                    split2(v[0], v[1], h0, l0);
                    split2(v[2], v[3], h1, l1);
                    const uint32_t at = piece(r, c & ~7) + static_cast<uint32_t>(c & 4) * 2;
#pragma unroll 4
                    for (int q = 0; q < p.width; ++q) {
                        st_cluster_b64(map_shared_rank(a_hi + at, q), h0, h1);
                        st_cluster_b64(map_shared_rank(a_lo + at, q), l0, l1);
                        if (on) st_cluster_f32(map_shared_rank(d_at + 4 * r, q), diagonal);
                    }
                }
            }
        }
        // ------------------------------------------------------------ square
        float o[32], d_row = 0.f;
        product(false, false, p.m, [&] {
            if (!mine) return;
            load_planes(a_hi, a_lo, row, c0, o);
            d_row = lds_f(d_at + 4 * row);
        });
        if (mine) {
            float v[32];
            sums_of(c0, v);
            const int q = shift_of(step);
            const float c3 = p.c3 * power_of_two(-2 * q), c5 = p.c5 * power_of_two(-4 * q);
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 d4 = lds128(d_at + 4 * (c0 + j));
                const float d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float& x = v[j + i];
                    if (c0 + j + i == row) {
                        sts_f(e_at + 4 * row, fmaf(c5, fmaf(d_row, d_row, x * 0x1p-24f), c3 * d_row));
                        x = 0.f;
                    } else {
                        x = fmaf(c5, fmaf(d_row + d[i], o[j + i], x * 0x1p-12f), c3 * o[j + i]);
                    }
                }
            }
            store_planes(a_hi, a_lo, row, c0, v);
        }
        // ------------------------------------------------------------ update
        float x[32], factor = 0.f;
        product(false, true, p.m, [&] {
            if (!active || c0 >= cols) return;
            load_planes(x_hi, x_lo, row, c0, x);
            factor = p.c1 + lds_f(e_at + 4 * row);
        });
        const bool last = step + 1 == p.steps;
        const int next = shift_of(step + 1);
        const float down = power_of_two(next - shift_of(step));
        factor *= down;
#pragma unroll 1
        for (int c = c0; active && c < cols; c += 32 * kSmallShare) {
            float v[32];
            if (c != c0) load_planes(x_hi, x_lo, row, c, x);
            sums_of(c, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = fmaf(factor, x[j], v[j] * (0x1p-12f * down));
            if (!last) {
                store_planes(x_hi, x_lo, row, c, v);
            } else if (row < p.m) {
                T* const out = static_cast<T*>(p.out) + e * p.so;
                const float result = 0x1p-13f * power_of_two(-next);
                if constexpr (TALL) {
                    T* o = out + (n0 + c) * p.ldo + row;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (c + j < cols) *o = from_f32<T>(v[j] * result);
                        o += p.ldo;
                    }
                } else {
                    T* const o = out + row * p.ldo + n0 + c;
                    if (p.align == 16 && c + 32 <= cols) {
#pragma unroll
                        for (int j = 0; j < 32; j += 16 / static_cast<int>(sizeof(T))) {
                            alignas(16) T y[16 / sizeof(T)];
#pragma unroll
                            for (int i = 0; i < 16 / static_cast<int>(sizeof(T)); ++i) y[i] = from_f32<T>(v[j + i] * result);
                            *reinterpret_cast<uint4*>(o + j) = *reinterpret_cast<const uint4*>(y);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (c + j < cols) o[j] = from_f32<T>(v[j] * result);
                    }
                }
            }
        }
    }

    if (timed_out) atomicOr(p.status, kGrStatusTimeout);
    __syncwarp();
    tc_fence_before_sync();
    if (p.width > 1)
        cluster_sync_all();  // (nobody writes to a CTA that has gone)
    else
        __syncthreads();
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc_cg<1>(tmem, S::kTmemCols);
    }
}

template <typename T, int W, int PARTS>
int set_up_width(int* most) {
    for (const auto kernel : {ortho_small_kernel<T, W, PARTS, false>, ortho_small_kernel<T, W, PARTS, true>}) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SmallShape<W, PARTS>::kSmem) != cudaSuccess)
            return SGEMM_ERR_CUDA;
        if (W == 256 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return SGEMM_ERR_CUDA;
    }
    if (W == 256) {  // whether the device holds clusters of 16
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(kSmallThreads);
        cfg.dynamicSmemBytes = SmallShape<W, PARTS>::kSmem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 16;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, ortho_small_kernel<T, W, PARTS, true>, &cfg) != cudaSuccess || clusters < 1) {
            (void)cudaGetLastError();
            *most = 8;
        }
    }
    return SGEMM_OK;
}

template <typename T, int W, int PARTS>
int launch(const OrthoCall& c, const OrthoSmallParams& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(c.E) * static_cast<unsigned>(p.width));
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = SmallShape<W, PARTS>::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(p.width);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = p.width > 1 ? 1 : 0;
    const auto kernel = c.M > c.N ? ortho_small_kernel<T, W, PARTS, true> : ortho_small_kernel<T, W, PARTS, false>;
    if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

template <typename T, int PARTS>
int set_up_type(int* most) {
    return set_up_width<T, 128, PARTS>(most) || set_up_width<T, 256, PARTS>(most);
}

template <typename T, int PARTS>
int launch_width(int w, const OrthoCall& c, const OrthoSmallParams& p, cudaStream_t s) {
    return w == 128 ? launch<T, 128, PARTS>(c, p, s) : launch<T, 256, PARTS>(c, p, s);
}

}  // namespace

int ortho_small_set_up(int* most_ctas) {
    *most_ctas = 16;
    if (set_up_type<float, 2>(most_ctas) || set_up_type<__nv_bfloat16, 2>(most_ctas) ||
        set_up_type<__nv_bfloat16, 1>(most_ctas) || set_up_type<__half, 2>(most_ctas)) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

int ortho_small(const OrthoCall& c, const DeviceState& st, cudaStream_t s) {
    const int m = std::min(c.M, c.N), n = std::max(c.M, c.N);
    // 128 columns a CTA in clusters of up to 8; 256 where one CTA then has all, or there are more.
    const int w = n <= 128 || (n > 256 && n <= 8 * 128) ? 128 : 256;
    if (m > 128 || n > 256 * st.ortho_ctas) return SGEMM_ERR_UNSUPPORTED;
    OrthoSmallParams p = {};
    const int size = c.type == SGEMM_TYPE_F32 ? 4 : 2;
    p.G = c.G, p.ldg = c.ldg, p.sg = c.sg, p.out = c.out, p.ldo = c.ldo, p.so = c.so;
    p.m = m, p.n = n, p.steps = c.steps, p.width = (n + w - 1) / w;
    p.vec = row_alignment(c.G, size, c.M > 1 ? c.ldg : 0, c.E > 1 ? c.sg : 0) == 16;
    p.align = row_alignment(c.out, size, c.M > 1 ? c.ldo : 0, c.E > 1 ? c.so : 0);
    p.c1 = c.a, p.c3 = c.b, p.c5 = c.c, p.growth = c.growth, p.eps = c.eps;
    p.timeout_ns = kDefaultTimeoutNs;
    p.status = st.status_word;
    if (c.type == SGEMM_TYPE_F32) return launch_width<float, 2>(w, c, p, s);
    if (c.type == SGEMM_TYPE_F16) return launch_width<__half, 2>(w, c, p, s);
    return c.parts == 2 ? launch_width<__nv_bfloat16, 2>(w, c, p, s) : launch_width<__nv_bfloat16, 1>(w, c, p, s);
}

}  // namespace detail
}  // namespace gb300
