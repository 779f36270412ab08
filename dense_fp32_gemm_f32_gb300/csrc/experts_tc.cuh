// Grouped products on the fifth-generation tensor cores (tcgen05): bf16 and
// f16 operands, float32 accumulation in tensor memory.
//
//     D[f, c] = sum_k A[f, k] B[c, k]
//
// The output's contiguous dimension f ("features") lies on the tensor core's
// 128 rows and the ragged dimension c on its columns, whose number an
// instruction sets in steps of 16.  So a group of 37 rows costs 48 columns and
// not a tile of 128, the weights stream through the operand that a decoding
// step fills anyway, and an accumulator row in a lane makes 32 lanes of a warp
// 32 neighbouring elements of an output row.
//
//   forward     f = output column n, c = row t of the group, k: A = W_e
//               (f innermost in HBM: MN-major), B = X (k innermost: K-major)
//   transposed  the same with A = W_e stored N x K (K-major)
//   gradient of the weights: f = n, c = k of X, contraction over the group's
//               rows t: A = dY, B = X, both MN-major, read as stored
//
// float32 operands come as three bf16 parts each, x = x0 + x1 + x2 (8 bits
// each, rounded to nearest: what is left is below 2^-25 |x|), and the sum runs
// over the six products of parts whose error a float32 product would show,
// smallest first; the three dropped ones are below 2^-24 |a||b| together.
//
// Persistent CTAs (CG = 1) or CTA pairs (CG = 2: one instruction of the pair's
// first CTA multiplies 256 features by up to 256 columns, each CTA holding
// half of either operand, which halves the shared-memory fill per flop).
// Tile i goes to cluster i mod clusters; which expert's rows it falls on every
// warp finds from the boundary array by itself (group_find), so the host
// never needs the group sizes.  Warps:
//   warp 0      loads: tensor-map copies of 64 k of A and B into a ring;
//   warp 1      MMAs (the pair's first CTA).  For a weight gradient the warp
//               first zeroes, in either CTA's shared memory, the rows past the
//               group's end in the slice that holds them: they are the next
//               group's, and may hold anything;
//   warps 2..5  epilogue: tensor memory -> registers -> HBM, while the MMAs of
//               the next tile fill the other accumulator.
//
// Every wait is bounded by `timeout_ns`; on expiry the thread records the
// timeout in the status word and goes to the final barrier.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "experts_groups.cuh"
#include "ptx.cuh"

namespace gb300 {

constexpr int kGrBK = 64;                // contraction per ring stage (128 bytes of 16-bit values)
constexpr int kGrThreads = 192;          // producer warp, MMA warp, 4 epilogue warps
constexpr unsigned int kGrStatusTimeout = 4u;  // the library's timeout bit

struct GroupedTcParams {
    const int* offsets;
    int T, E;
    int wgrad;          // 0: the group's rows are columns c; 1: they are the contraction
    int F, C, K;        // features; wgrad: columns; forward: contraction length
    int ftiles, ctiles; // feature tiles; wgrad: column tiles
    int nseg;           // products of parts summed: 1, or 6 for float32
    int a_planes;       // third coordinate of A's part p, expert e: p * a_planes + (wgrad ? 0 : e)
    void* out;
    long long ldo, so;  // elements between rows; wgrad: between experts
    int out_type;
    uint32_t idesc;     // instruction descriptor without the column count
    unsigned long long timeout_ns;
    unsigned int* status;
};

// Parts of A and B in each of float32's six products.
__device__ __forceinline__ int seg_a(int seg) { return (0x210100 >> (4 * (5 - seg))) & 15; }
__device__ __forceinline__ int seg_b(int seg) { return (0x012010 >> (4 * (5 - seg))) & 15; }

template <int TN_, int CG_>
struct GroupedShape {
    static constexpr int TN = TN_, CG = CG_;
    static constexpr int kABytes = 128 * 128;        // 128 features x 64 k
    static constexpr int kBBytes = TN / CG * 128;    // this CTA's columns x 64 k
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = (200 * 1024) / kStageBytes;
    static constexpr int kAccCols = TN < 32 ? 32 : TN;
    static constexpr int kTmemCols = 2 * kAccCols;
    static constexpr int kBars = 3 * kStages + 4;    // full, empty, peer_full; acc_full, acc_empty x 2
    static constexpr int kSmem = kStages * kStageBytes + 8 * kBars + 16 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory columns");
};

struct GroupedTile {
    int e, f0, c0, cols, k0, klen;  // c0: row t (forward) or column of X; k0: first row of the contraction (wgrad)
};

// Tile number `i`, from the same cursor in increasing order.
template <int TN, int FT>
__device__ __forceinline__ bool grouped_tile(const GroupedTcParams& p, int i, GroupCursor& cur, GroupedTile& t) {
    GroupHit h;
    if (p.wgrad) {
        const int per = p.ftiles * p.ctiles;
        if (!group_find(p.offsets, p.E, p.T, i, cur, [&](int) { return per; }, h)) return false;
        t.f0 = h.local / p.ctiles * FT;
        t.c0 = h.local % p.ctiles * TN;
        t.cols = min(TN, p.C - t.c0);
        t.k0 = h.start;
        t.klen = h.end - h.start;
    } else {
        if (!group_find(p.offsets, p.E, p.T, i, cur, [&](int n) { return (n + TN - 1) / TN * p.ftiles; }, h))
            return false;
        const int n = (h.end - h.start + TN - 1) / TN;
        t.f0 = h.local / n * FT;
        t.c0 = h.start + h.local % n * TN;
        t.cols = min(TN, h.end - t.c0);
        t.k0 = 0;
        t.klen = p.K;
    }
    t.e = h.e;
    return true;
}

// A weight gradient's slice with `left` rows from its first to the group's end
// whose last instruction takes rows past that end.
__device__ __forceinline__ bool grouped_tail(int left) { return left < kGrBK && (left & 15) != 0; }

template <typename T>
__device__ __forceinline__ void grouped_store(void* out, long long at, long long ld, const uint32_t (&v)[32], int n,
                                              bool zero) {
    T* o = static_cast<T*>(out) + at;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        if (j < n) *o = from_f32<T>(zero ? 0.f : __uint_as_float(v[j]));
        o += ld;
    }
}

// Rows of no expert: zeros, spread over the CTAs' epilogue warps.
template <typename T>
__device__ void grouped_zero_rows(const GroupedTcParams& p, int worker, int workers) {
    const int lane = threadIdx.x & 31;
    const int first = group_bound(p.offsets, 0, p.T);
    int last = first;
    for (int i = lane; i <= p.E; i += 32) last = max(last, group_bound(p.offsets, i, p.T));
    last = __reduce_max_sync(0xffffffffu, last);
    const int rows = first + (p.T - last);
    for (int r = worker; r < rows; r += workers) {
        T* o = static_cast<T*>(p.out) + static_cast<long long>(r < first ? r : last + r - first) * p.ldo;
        for (int f = lane; f < p.F; f += 32) o[f] = from_f32<T>(0.f);
    }
}

// AMN, BMN: the operand is MN-major in HBM and shared memory (else K-major).
template <bool AMN, bool BMN, int TN, int CG>
__global__ void __launch_bounds__(kGrThreads, 1)
    grouped_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const GroupedTcParams p) {
    using S = GroupedShape<TN, CG>;
    constexpr int FT = 128 * CG;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    auto sA = [&](int s) { return base + static_cast<uint32_t>(s * S::kStageBytes); };
    auto sB = [&](int s) { return sA(s) + S::kABytes; };
    const uint32_t bars = base + S::kStages * S::kStageBytes;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (S::kStages + s); };
    auto peer_full = [&](int s) { return bars + 8u * (2 * S::kStages + s); };
    auto acc_full = [&](int b) { return bars + 8u * (3 * S::kStages + b); };
    auto acc_empty = [&](int b) { return bars + 8u * (3 * S::kStages + 2 + b); };
    const uint32_t tmem_slot = bars + 8u * S::kBars;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0;
    const int cluster = static_cast<int>(blockIdx.x) / CG, clusters = static_cast<int>(gridDim.x) / CG;
    const unsigned long long tmo = p.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
            mbar_init(peer_full(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), 4 * CG);
        }
        fence_mbarrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, S::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync_all();  // the peer's barriers are ready
    tc_fence_after_sync();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot) : "memory");

    bool timed_out = false;
    GroupCursor cur = group_begin(p.offsets, p.T);
    GroupedTile t;
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        int it = 0;  // ring position, over all tiles
        for (int i = cluster; !timed_out && grouped_tile<TN, FT>(p, i, cur, t); i += clusters) {
            const int nk = (t.klen + kGrBK - 1) / kGrBK;
            const int cols = (t.cols + 15) & ~15;            // columns of the instruction,
            const int mine = CG == 2 ? cols / 2 : cols;      // this CTA's part of them
            const int c0 = t.c0 + static_cast<int>(rank) * mine;
            const int f0 = t.f0 + static_cast<int>(rank) * 128;
            const int boxes = BMN ? (mine + 63) / 64 : (mine + 31) / 32;
            constexpr int kBox = BMN ? 64 * 128 : 32 * 128;
            if (lane == 0) {
                for (int seg = 0; seg < p.nseg && !timed_out; ++seg) {
                    const int pa = (p.nseg > 1 ? seg_a(seg) : 0) * p.a_planes + (p.wgrad ? 0 : t.e);
                    const int pb = p.nseg > 1 ? seg_b(seg) : 0;
                    for (int kt = 0; kt < nk; ++kt, ++it) {
                        const int s = it % S::kStages, round = it / S::kStages;
                        if (round > 0 && !mbar_wait_spin<CG == 2>(empty(s), (round - 1) & 1, tmo)) {
                            timed_out = true;
                            break;
                        }
                        const int k = t.k0 + kt * kGrBK;
                        // The pair's loads all arrive on the first CTA's
                        // barrier, but for a slice whose rows past the end
                        // the second CTA has to zero first.
                        const bool own = CG == 1 || (BMN && grouped_tail(t.klen - kt * kGrBK));
                        const uint32_t bar = own || rank == 0 ? full(s) : map_shared_rank(full(s), 0);
                        const uint32_t bytes = S::kABytes + boxes * kBox;
                        if (own || rank == 0) mbar_arrive_expect_tx(full(s), own ? bytes : 2 * bytes);
                        auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, int z) {
                            if constexpr (CG == 2)
                                tma_load_3d_pair(dst, map, bar, x, y, z);
                            else
                                tma_load_3d(dst, map, bar, x, y, z);
                        };
                        if constexpr (AMN) {
                            load(sA(s), &tmA, f0, k, pa);
                            load(sA(s) + 64 * 128, &tmA, f0 + 64, k, pa);
                        } else {
                            load(sA(s), &tmA, k, f0, pa);
                        }
                        for (int b = 0; b < boxes; ++b) {
                            if constexpr (BMN)
                                load(sB(s) + b * kBox, &tmB, c0 + 64 * b, k, pb);
                            else
                                load(sB(s) + b * kBox, &tmB, k, c0 + 32 * b, pb);
                        }
                    }
                }
            }
            it = __shfl_sync(0xffffffffu, it, 0);
            timed_out = __shfl_sync(0xffffffffu, timed_out ? 1 : 0, 0) != 0;
        }
        // (every copy lands before its CTA ends: the MMAs wait for it, and the
        // epilogue for them; after a timeout, the wait below, in the first CTA
        // for the pair)
        if (timed_out && rank == 0 && lane == 0)
            for (int j = max(0, it - S::kStages); j < it; ++j)
                (void)mbar_wait_spin<CG == 2>(full(j % S::kStages), (j / S::kStages) & 1, tmo);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        int it = 0, tile = 0;
        int tails = 0;  // bit s: parity of such slices so far in stage s
        for (int i = cluster; !timed_out && grouped_tile<TN, FT>(p, i, cur, t); i += clusters, ++tile) {
            const int nk = (t.klen + kGrBK - 1) / kGrBK;
            const int cols = (t.cols + 15) & ~15;
            const int buf = tile & 1;
            const uint32_t acc = tmem + static_cast<uint32_t>(buf * S::kAccCols);
            const uint32_t idesc = p.idesc | static_cast<uint32_t>(cols >> 3) << 17;
            if (rank == 0 && tile >= 2) {
                if (!__all_sync(0xffffffffu, mbar_wait_spin<CG == 2>(acc_empty(buf), ((tile >> 1) - 1) & 1, tmo))) {
                    timed_out = true;
                    break;
                }
                tc_fence_after_sync();
            }
            for (int n = 0; n < p.nseg * nk && !timed_out; ++n, ++it) {
                const int kt = n % nk;
                const int s = it % S::kStages, phase = (it / S::kStages) & 1;
                const int left = t.klen - kt * kGrBK;  // of the contraction, from this slice on
                const bool tail = BMN && grouped_tail(left);
                if (rank != 0 && !tail) continue;  // (the first CTA waits for this one's loads)
                // (the second CTA's barriers see such slices' loads only)
                const int full_phase = rank != 0 ? tails >> s & 1 : phase;
                if (!__all_sync(0xffffffffu, mbar_wait_spin<CG == 2>(full(s), full_phase, tmo))) {
                    timed_out = true;
                    break;
                }
                if constexpr (BMN) {
                    // Rows left .. of the last instruction's 16 belong to
                    // others: zeros (rows of 128 bytes in blocks of 64 rows).
                    if (tail) {
                        const int past = (left + 15) & ~15;
                        const int blocks = 2 + S::kBBytes / (64 * 128);  // A's and B's
                        for (int j = lane; j < blocks * (past - left) * 8; j += 32) {
                            const int q = j & 7, row = left + (j >> 3) % (past - left), b = (j >> 3) / (past - left);
                            sts128(sA(s) + static_cast<uint32_t>(b * 64 * 128 + row * 128 + q * 16),
                                   make_float4(0.f, 0.f, 0.f, 0.f));
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if constexpr (CG == 2) {
                            const int tail_phase = tails >> s & 1;
                            tails ^= 1 << s;
                            if (rank != 0) {
                                if (lane == 0) mbar_arrive_cluster(map_shared_rank(peer_full(s), 0));
                                continue;
                            }
                            if (!__all_sync(0xffffffffu, mbar_wait_spin<true>(peer_full(s), tail_phase, tmo))) {
                                timed_out = true;
                                break;
                            }
                        }
                    }
                }
                tc_fence_after_sync();
                if (lane == 0) {
                    const uint64_t da = AMN ? umma_desc_mnmajor_sw128(sA(s), 64 * 128) : umma_desc_kmajor_sw128(sA(s));
                    const uint64_t db = BMN ? umma_desc_mnmajor_sw128(sB(s), 64 * 128) : umma_desc_kmajor_sw128(sB(s));
                    // 16 k: 32 bytes of each row (K-major), 16 rows of 128 bytes (MN-major); addresses in units of 16
                    constexpr uint64_t ka = AMN ? 128 : 2, kb = BMN ? 128 : 2;
#pragma unroll
                    for (int kk = 0; kk < kGrBK / 16; ++kk)
                        if (kk * 16 < left) umma_f16<CG>(acc, da + kk * ka, db + kk * kb, idesc, n > 0 || kk > 0);
                    umma_commit_cg<CG>(empty(s));
                    if constexpr (CG == 2) umma_commit_cg<CG>(map_shared_rank(empty(s), 1));
                }
                __syncwarp();
            }
            if (rank == 0 && !timed_out && lane == 0) {
                umma_commit_cg<CG>(acc_full(buf));
                if constexpr (CG == 2) umma_commit_cg<CG>(map_shared_rank(acc_full(buf), 1));
            }
            __syncwarp();
        }
        if (timed_out && rank == 0 && lane == 0) {  // the MMAs in flight end before tensor memory is freed
            umma_commit_cg<CG>(acc_full(tile & 1));
            (void)mbar_wait_spin<CG == 2>(acc_full(tile & 1), (tile >> 1) & 1, tmo);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;
        if (!p.wgrad) {
            const int worker = static_cast<int>(blockIdx.x) * 4 + q, workers = static_cast<int>(gridDim.x) * 4;
            if (p.out_type == 0)
                grouped_zero_rows<float>(p, worker, workers);
            else  // (bf16 and f16 zeros are the same bits)
                grouped_zero_rows<__half>(p, worker, workers);
        }
        int tile = 0;
        for (int i = cluster; grouped_tile<TN, FT>(p, i, cur, t); i += clusters, ++tile) {
            const int buf = tile & 1;
            if (!__all_sync(0xffffffffu, mbar_wait_spin<CG == 2>(acc_full(buf), (tile >> 1) & 1, tmo))) {
                timed_out = true;
                break;
            }
            tc_fence_after_sync();
            const uint32_t acc =
                tmem + static_cast<uint32_t>(buf * S::kAccCols) + (static_cast<uint32_t>(32 * q) << 16);
            const int f = t.f0 + static_cast<int>(rank) * 128 + 32 * q + lane;
            const bool zero = t.klen == 0;  // no MMA wrote the accumulator
            for (int c = 0; c < t.cols; c += 32) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(c), v);
                tmem_wait_ld();
                const long long at = (p.wgrad ? t.e * p.so : 0ll) + (t.c0 + c) * p.ldo + f;
                const int n = f < p.F ? t.cols - c : 0;
                if (p.out_type == 0)
                    grouped_store<float>(p.out, at, p.ldo, v, n, zero);
                else if (p.out_type == 1)
                    grouped_store<__nv_bfloat16>(p.out, at, p.ldo, v, n, zero);
                else
                    grouped_store<__half>(p.out, at, p.ldo, v, n, zero);
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (CG == 1 || rank == 0)
                    mbar_arrive(acc_empty(buf));
                else
                    mbar_arrive_cluster(map_shared_rank(acc_empty(buf), 0));
            }
        }
    }

    if (timed_out) atomicOr(p.status, kGrStatusTimeout);
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync_all();  // nothing of the peer's is under way in this CTA's memory
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_cg<CG>(tmem, S::kTmemCols);
    }
}

}  // namespace gb300
