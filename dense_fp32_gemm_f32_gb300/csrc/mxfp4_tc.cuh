// Products of MXFP4 operands on the fifth-generation tensor cores, dense and
// grouped by expert: the layout, tiles, roles and schedule of experts_tc.cuh
// (features on the 128 rows, ragged rows on the columns; A = the weights, B =
// the rows, both K-major) with block-scaled 4-bit instructions.
//
//     D[f, c] = sum over blocks b of 32 k: 2^(sa[f,b] + sb[c,b]) sum_k a[f, k] b[c, k]
//
// A ring stage is 256 k: 128 bytes of codes a row, as the tensor maps and the
// swizzle take them, and 8 scales a row.  The scale blocks in HBM (128 rows x 4
// scales, 512 bytes) are what tcgen05.cp spreads over 4 tensor-memory columns
// as the instructions read them: row r's 4 bytes in lane r mod 32, column r / 32.
// So scales go HBM -> shared memory (as 32-bit boxes of 256: the only copies
// that may signal a pair's other CTA are tensor-map copies) -> tensor memory
// without a thread touching them.  An instruction takes 64 k and, through its descriptor, one half of the
// 4 bytes.
//
// The wide tile (256 features x 256 columns a CTA pair) fills half of tensor
// memory and the scales need some of the rest, so it has one accumulator; its 8
// epilogue warps take it whole into registers before they store, and the next
// tile's MMAs start after the reading (about 1/20 of the MMAs of K = 4096)
// and not after the stores.
#pragma once

#include "experts_tc.cuh"

namespace gb300 {

constexpr int kMxBK = 256;  // contraction per ring stage (128 bytes of codes)

struct Mxfp4TcParams {
    const int* offsets;  // null: one group of all T rows
    int T, E;
    int F, K;            // features, contraction (a multiple of 32)
    int ftiles;
    void* out;
    long long ldo;
    int out_type;
    unsigned long long timeout_ns;
    unsigned int* status;
};

template <int TN_, int CG_>
struct Mxfp4Shape {
    static constexpr int TN = TN_, CG = CG_;
    static constexpr int kCols = TN / CG;
    static constexpr int kABytes = 128 * 128;
    static constexpr int kBBytes = kCols * 128;
    static constexpr int kSbBlocks = (TN + 127) / 128;         // scale row blocks of the columns
    static constexpr int kSaBytes = 1024, kSbBytes = 1024 * kSbBlocks;
    static constexpr int kStageBytes = kABytes + kBBytes + kSaBytes + kSbBytes;
    static constexpr int kStages = (218 * 1024) / kStageBytes < 10 ? (218 * 1024) / kStageBytes : 10;
    static constexpr int kBoxCols = kCols < 64 ? kCols : 64;
    static constexpr int kAccs = TN > 128 ? 1 : 2;              // accumulators
    static constexpr int kScaleCol = kAccs * TN;                // tensor-memory column of the scales
    static constexpr int kTmemUsed = kScaleCol + 2 * (4 + 4 * kSbBlocks);
    static constexpr int kTmemCols = kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
    static constexpr int kEpilogueWarps = TN > 128 ? 8 : 4;
    static constexpr int kThreads = 64 + 32 * kEpilogueWarps;
    static constexpr int kBars = 2 * kStages + 4;               // full, empty; acc_full, acc_empty x 2
    static constexpr int kSmem = kStages * kStageBytes + 8 * kBars + 16 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(kStageBytes % 1024 == 0, "operand tiles start on the swizzle's 1024 bytes");
    static_assert(kTmemUsed <= 512, "tensor memory columns");
};

struct Mxfp4Tile {
    int e, f0, c0, cols;
    int srow;  // the first column's place among the scale blocks' rows
};

template <int TN, int FT>
__device__ __forceinline__ bool mxfp4_tile(const Mxfp4TcParams& p, int i, GroupCursor& cur, Mxfp4Tile& t) {
    int start = 0, end = p.T, local = i, block0 = 0, e = 0;
    if (p.offsets) {
        GroupHit h;
        if (!group_find(p.offsets, p.E, p.T, i, cur, [&](int n) { return (n + TN - 1) / TN * p.ftiles; }, h))
            return false;
        start = h.start, end = h.end, local = h.local, block0 = h.block0, e = h.e;
    } else if (i >= (p.T + TN - 1) / TN * p.ftiles) {
        return false;
    }
    const int n = (end - start + TN - 1) / TN;
    const int off = local % n * TN;
    t.e = e;
    t.f0 = local / n * FT;
    t.c0 = start + off;
    t.cols = min(TN, end - t.c0);
    t.srow = 128 * block0 + off;
    return true;
}

template <int TN, int CG>
__global__ void __launch_bounds__(Mxfp4Shape<TN, CG>::kThreads, 1)
    mxfp4_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSa, const __grid_constant__ CUtensorMap tmSb,
                    const Mxfp4TcParams p) {
    using S = Mxfp4Shape<TN, CG>;
    constexpr int FT = 128 * CG;
    constexpr bool PAIR = CG == 2;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t baseB = base + S::kABytes, baseSa = baseB + S::kBBytes, baseSb = baseSa + S::kSaBytes;
    const uint32_t bars = base + S::kStages * S::kStageBytes;
    const uint32_t full0 = bars, empty0 = bars + 8 * S::kStages;
    const uint32_t acc_full0 = bars + 16 * S::kStages, acc_empty0 = acc_full0 + 16;
    const uint32_t tmem_slot = bars + 8u * S::kBars;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
    const int cluster = static_cast<int>(blockIdx.x) / CG, clusters = static_cast<int>(gridDim.x) / CG;
    const unsigned long long tmo = p.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < S::kAccs; ++b) {
            mbar_init(acc_full0 + 8 * b, 1);
            mbar_init(acc_empty0 + 8 * b, S::kEpilogueWarps * CG);
        }
        fence_mbarrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, S::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();
    tc_fence_after_sync();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot) : "memory");

    bool timed_out = false;
    GroupCursor cur = p.offsets ? group_begin(p.offsets, p.T) : GroupCursor();
    Mxfp4Tile t;
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        const uint32_t bar0 = PAIR && rank != 0 ? map_shared_rank(full0, 0) : full0;
        uint32_t s = 0, phase = 1;
        int issued = 0;
        for (int i = cluster; !timed_out && mxfp4_tile<TN, FT>(p, i, cur, t); i += clusters) {
            const int mine = ((t.cols + 15) & ~15) / CG;
            const int c0 = t.c0 + rank * mine, f0 = t.f0 + rank * 128;
            const int boxes = (mine + S::kBoxCols - 1) / S::kBoxCols;
            constexpr uint32_t kBox = S::kBoxCols * 128;
            const uint32_t bytes = S::kABytes + boxes * kBox + S::kSaBytes + S::kSbBytes;
            if (lane == 0) {
                for (int k = 0; k < p.K; k += kMxBK) {
                    if (!mbar_wait_spin<false>(empty0 + 8 * s, phase, tmo)) {
                        timed_out = true;
                        break;
                    }
                    const uint32_t bar = bar0 + 8 * s;
                    const uint32_t st = s * S::kStageBytes;
                    auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, int z) {
                        if constexpr (PAIR)
                            tma_load_3d_pair(dst, map, bar, x, y, z);
                        else
                            tma_load_3d(dst, map, bar, x, y, z);
                    };
                    if (rank == 0) mbar_arrive_expect_tx(bar, CG * bytes);
                    load(base + st, &tmA, k >> 1, f0, t.e);
#pragma unroll 1
                    for (int j = 0; j < boxes; ++j)
                        load(baseB + st + j * kBox, &tmB, k >> 1, c0 + S::kBoxCols * j, 0);
                    // (words; the 8 scales of 256 k are 1024 bytes of 128 rows)
                    load(baseSa + st, &tmSa, k, f0 >> 7, t.e);
                    load(baseSb + st, &tmSb, k, t.srow >> 7, 0);
                    ++issued;
                    if (++s == S::kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            timed_out = __any_sync(0xffffffffu, timed_out);
        }
        if (timed_out && rank == 0 && lane == 0)
            for (int j = max(0, issued - S::kStages); j < issued; ++j)
                (void)mbar_wait_spin<false>(full0 + 8 * (j % S::kStages), (j / S::kStages) & 1, tmo);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        const uint64_t descA = umma_desc_kmajor_sw128(base), descB = umma_desc_kmajor_sw128(baseB);
        const uint64_t descSa = umma_desc_rows16(baseSa), descSb = umma_desc_rows16(baseSb);
        const uint32_t sfa = tmem + S::kScaleCol, sfb = sfa + 8;
        const uint32_t peer_empty0 = PAIR ? map_shared_rank(empty0, 1) : 0;
        const uint32_t peer_acc_full0 = PAIR ? map_shared_rank(acc_full0, 1) : 0;
        // float32 accumulator, e2m1 x e2m1, e8m0 scales, M
        constexpr uint32_t kIdesc = 1u << 7 | 1u << 10 | 1u << 23 | static_cast<uint32_t>(FT / 16) << 24;
        uint32_t s = 0, phase = 0;
        int unit = 0;
        for (int i = cluster; !timed_out && mxfp4_tile<TN, FT>(p, i, cur, t); i += clusters, ++unit) {
            const int buf = unit % S::kAccs, round = unit / S::kAccs;
            const uint32_t acc = tmem + static_cast<uint32_t>(buf * TN);
            const uint32_t idesc = kIdesc | static_cast<uint32_t>((t.cols + 15) >> 4) << 18;
            const uint32_t sb_col = sfb + ((t.srow & 127) >> 5);  // (32 rows of scales a column)
            if (rank == 0 && lane == 0) {
                if (round > 0 && !mbar_wait_spin<PAIR>(acc_empty0 + 8 * buf, (round - 1) & 1, tmo)) timed_out = true;
                tc_fence_after_sync();
                for (int k = 0; k < p.K && !timed_out; k += kMxBK) {
                    if (!mbar_wait_spin<false>(full0 + 8 * s, phase, tmo)) {
                        timed_out = true;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t off = s * (S::kStageBytes / 16);
                    const uint64_t a = descA + off, b = descB + off, ca = descSa + off, cb = descSb + off;
                    const int left = p.K - k;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // 128 k: one scale block of each row block
                        if (left > 128 * h) {
                            tmem_cp_32x128b_x4<CG>(sfa + 4 * h, ca + 32 * h);
#pragma unroll
                            for (int j = 0; j < S::kSbBlocks; ++j)
                                tmem_cp_32x128b_x4<CG>(sfb + 4 * (S::kSbBlocks * h + j), cb + 64 * j + 32 * h);
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk)  // 64 k: scales 0, 1 or 2, 3 of the block
                                if (left > 128 * h + 64 * kk)
                                    umma_mxf4<CG>(acc, a + 4 * h + 2 * kk, b + 4 * h + 2 * kk,
                                                  idesc | (kk ? 2u << 4 | 2u << 29 : 0u), sfa + 4 * h,
                                                  sb_col + 4 * S::kSbBlocks * h, k > 0 || h > 0 || kk > 0);
                        }
                    }
                    umma_commit_cg<CG>(empty0 + 8 * s);
                    if constexpr (PAIR) umma_commit_cg<CG>(peer_empty0 + 8 * s);
                    if (++s == S::kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
                if (!timed_out) {
                    umma_commit_cg<CG>(acc_full0 + 8 * buf);
                    if constexpr (PAIR) umma_commit_cg<CG>(peer_acc_full0 + 8 * buf);
                }
            }
            timed_out = __any_sync(0xffffffffu, timed_out);
            if (timed_out) break;
        }
        if (timed_out && rank == 0 && lane == 0) {
            const int buf = unit % S::kAccs, round = unit / S::kAccs;
            umma_commit_cg<CG>(acc_full0 + 8 * buf);
            (void)mbar_wait_spin<false>(acc_full0 + 8 * buf, round & 1, tmo);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;
        constexpr int kMine = TN / (S::kEpilogueWarps / 4);  // columns of this warp
        const int mine0 = (warp - 2) / 4 * kMine;
        const uint32_t acc_empty_lead = PAIR && rank != 0 ? map_shared_rank(acc_empty0, 0) : acc_empty0;
        if (p.offsets) {
            GroupedTcParams z;  // (the fields that the zeroing reads)
            z.offsets = p.offsets, z.T = p.T, z.E = p.E, z.F = p.F, z.out = p.out, z.ldo = p.ldo;
            const int worker = static_cast<int>(blockIdx.x) * S::kEpilogueWarps + warp - 2;
            const int workers = static_cast<int>(gridDim.x) * S::kEpilogueWarps;
            if (p.out_type == 0)
                grouped_zero_rows<float>(z, worker, workers);
            else
                grouped_zero_rows<__half>(z, worker, workers);
        }
        int unit = 0;
        for (int i = cluster; mxfp4_tile<TN, FT>(p, i, cur, t); i += clusters, ++unit) {
            const int buf = unit % S::kAccs, round = unit / S::kAccs;
            if (!__all_sync(0xffffffffu, mbar_wait_spin<false>(acc_full0 + 8 * buf, round & 1, tmo))) {
                timed_out = true;
                break;
            }
            tc_fence_after_sync();
            const uint32_t acc = tmem + static_cast<uint32_t>(buf * TN + mine0) + (static_cast<uint32_t>(32 * q) << 16);
            uint32_t v[kMine / 32][32];
#pragma unroll
            for (int c = 0; c < kMine / 32; ++c)
                if (mine0 + 32 * c < t.cols) tmem_ld_32x32b_x32(acc + 32 * c, v[c]);
            tmem_wait_ld();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (!PAIR || rank == 0)
                    mbar_arrive(acc_empty0 + 8 * buf);
                else
                    mbar_arrive_cluster(acc_empty_lead + 8 * buf);
            }
            const int f = t.f0 + rank * 128 + 32 * q + lane;
            const int cols = (f < p.F ? t.cols : 0) - mine0;
            void* const out = p.out;
            const long long at = static_cast<long long>(t.c0 + mine0) * p.ldo + f;
#pragma unroll
            for (int c = 0; c < kMine / 32; ++c) {
                if (mine0 + 32 * c < t.cols) {
                    const long long o = at + 32 * c * p.ldo;
                    if (p.out_type == 0)
                        grouped_store<float>(out, o, p.ldo, v[c], cols - 32 * c);
                    else if (p.out_type == 1)
                        grouped_store<__nv_bfloat16>(out, o, p.ldo, v[c], cols - 32 * c);
                    else
                        grouped_store<__half>(out, o, p.ldo, v[c], cols - 32 * c);
                }
            }
        }
    }

    if (timed_out) atomicOr(p.status, kGrStatusTimeout);
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_cg<CG>(tmem, S::kTmemCols);
    }
}

}  // namespace gb300
