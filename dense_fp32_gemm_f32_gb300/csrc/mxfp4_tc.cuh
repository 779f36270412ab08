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
// The wide tile has 192 columns and not 256: two accumulators of 256 would fill
// tensor memory and leave the scales no room, and with one accumulator the
// MMAs wait for the epilogue to empty it, 1.5 us a tile.  (Either way 155 us
// for 16384 rows, 8 experts of 8192 x 4096, where the smaller tile's loads cost
// what the overlap saves; 4096 x 4096 x 8192 43 and 40 us.)  7.1 PFLOP/s; with the
// loads switched off 126 us, the MMAs' own time, with the MMAs off 136.  One row
// x 8192 x 8192, 64 tiles shared by two CTAs each: 7.6 us, 4.7 TB/s.  Tiles are
// multiples of 64 columns, so that a tile's scales begin 0 or 2 tensor-memory
// columns into their block: B's scales have to begin at an even column.
#pragma once

#include "experts_tc.cuh"

namespace gb300 {

constexpr int kMxBK = 256;  // contraction per ring stage (128 bytes of codes)

// Contraction after which the accumulators go to float32 registers.  Measured: an
// instruction (64 k) cuts the sum to 24 bits, so that 256 of them stay below
// 256 * 2^-23 = 3.1e-5 of the sum of magnitudes.  (One accumulator for all of 65536,
// a block of both rows 2^10 times the others: 6.4e-5; 262144, magnitudes within
// 2^12 of one another: 9.4e-5.)
constexpr int kMxChunk = 16384;

struct Mxfp4TcParams {
    const int* offsets;  // null: one group of all T rows
    int T, E;
    int F, K;            // features, contraction (a multiple of 32)
    int ftiles;
    void* out;
    long long ldo;
    int out_type;
    int align;
    int ks;  // SPLIT: CTAs of a cluster
    unsigned long long timeout_ns;
    unsigned int* status;
};

// LONG: a contraction of more than kMxChunk.
template <int TN_, int CG_, bool LONG = false>
struct Mxfp4Shape {
    static constexpr int TN = TN_, CG = CG_;
    static constexpr int kCols = TN / CG;
    static constexpr int kABytes = 128 * 128;
    static constexpr int kBBytes = kCols * 128;
    static constexpr int kBoxCols = kCols / 2;                  // columns of a tensor-map box of B
    // Scale row blocks of a tile's columns, which begin 0 or 64 rows into one.
    static constexpr int kSbBlocks = (TN + 64 + 127) / 128;
    static constexpr int kSaBytes = 1024, kSbBytes = 1024 * kSbBlocks;
    static constexpr int kStageBytes = kABytes + kBBytes + kSaBytes + kSbBytes;
    static constexpr int kScaleCol = 2 * TN;                       // tensor-memory column of the scales
    static constexpr int kScaleCols = 2 * (4 + 4 * kSbBlocks);     // of a stage; two stages take turns
    static constexpr int kTmemUsed = kScaleCol + 2 * kScaleCols;
    static constexpr int kTmemCols = kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
    // (8 for the wide tile: 159 us instead of 157, as above; but 4 have no registers for its
    // sums.  LONG for 4096 x 4096 x 32768: 158 us, 153 with one accumulator.)
    static constexpr int kEpiWarps = LONG && TN > 64 ? 8 : 4;
    static constexpr int kThreads = 32 * (3 + kEpiWarps);
    static constexpr int kPatches = kEpiWarps * kGrPatchBytes;
    static constexpr int kStages = kRing(kStageBytes, kPatches);
    static constexpr int kBars = 2 * kStages + 4 + kSchedBars;  // full, empty; acc_full, acc_empty x 2
    static constexpr int kSmem = kStages * kStageBytes + kPatches + kSchedBytes + 8 * kBars + 16 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(TN % 128 == 64 && kCols % 8 == 0 && kBoxCols % 8 == 0 && kCols % kBoxCols == 0, "tile");
    static_assert(kStageBytes % 1024 == 0 && kBBytes % 1024 == 0, "operand tiles start on the swizzle's 1024 bytes");
    static_assert(kTmemUsed <= 512, "tensor memory columns");
    static_assert(kBoxCols * 128 % 1024 == 0, "boxes start on the swizzle's 1024 bytes");
};

template <int TN>
__device__ __forceinline__ int mxfp4_tiles(const Mxfp4TcParams& p) {
    auto units = [&](int n) { return (n + TN - 1) / TN * p.ftiles; };
    return p.offsets ? group_total(p.offsets, p.E, p.T, units) : units(p.T);
}

template <int TN, int FT>
__device__ __forceinline__ void mxfp4_tile(const Mxfp4TcParams& p, int i, GroupCursor& cur, GroupedTile& t) {
    GroupHit h = {0, 0, p.T, i, 0};
    if (p.offsets)
        (void)group_find(p.offsets, p.E, p.T, i, cur, [&](int n) { return (n + TN - 1) / TN * p.ftiles; }, h);
    const int n = max(1, (h.end - h.start + TN - 1) / TN);
    int f, row;
    tile_place(h.local, n, p.ftiles, f, row);
    const int off = row * TN;
    t.e = h.e;
    t.f0 = f * FT;
    t.c0 = h.start + off;
    t.cols = min(TN, h.end - t.c0);
    t.k0 = 0;
    t.klen = p.K;
    t.srow = 128 * h.block0 + off;
}

// SPLIT: as in grouped_tc_kernel.
template <int TN, int CG, bool SPLIT = false, bool LONG = false>
__global__ void __launch_bounds__(Mxfp4Shape<TN, CG, LONG>::kThreads, 1)
    mxfp4_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSa, const __grid_constant__ CUtensorMap tmSb,
                    const Mxfp4TcParams p) {
    using S = Mxfp4Shape<TN, CG, LONG>;
    constexpr int FT = 128 * CG;
    constexpr bool PAIR = CG == 2;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t baseB = base + S::kABytes, baseSa = baseB + S::kBBytes, baseSb = baseSa + S::kSaBytes;
    const uint32_t patches = base + S::kStages * S::kStageBytes;
    const uint32_t slots = patches + S::kPatches;
    const uint32_t bars = slots + kSchedBytes;
    const uint32_t full0 = bars, empty0 = bars + 8 * S::kStages;
    const uint32_t acc_full0 = bars + 16 * S::kStages, acc_empty0 = acc_full0 + 16, sched0 = acc_empty0 + 16;
    const uint32_t tmem_slot = bars + 8u * S::kBars;

    const int warp = warp_uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int rank = PAIR ? warp_uniform(static_cast<int>(cluster_ctarank())) : 0;
    static_assert(!SPLIT || (CG == 1 && S::kStages * S::kStageBytes >= TN * 128 * 4), "split form");
    const int share = SPLIT ? p.ks : CG;
    const int part = SPLIT ? warp_uniform(static_cast<int>(cluster_ctarank())) : 0;
    const int cluster = static_cast<int>(blockIdx.x) / share, clusters = static_cast<int>(gridDim.x) / share;
    const unsigned long long tmo = p.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full0 + 8 * b, 1);
            mbar_init(acc_empty0 + 8 * b, S::kEpiWarps * CG);
        }
        for (int j = 0; j < kSchedSlots; ++j) {
            mbar_init(sched0 + 8 * j, 1);
            mbar_init(sched0 + 8 * (kSchedSlots + j), 2 + S::kEpiWarps);
        }
        fence_mbarrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmSa);
        prefetch_tensormap(&tmSb);
    }
    __syncwarp();
    if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, S::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();
    tc_fence_after_sync();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot) : "memory");
    tmem = warp_uniform(tmem);
    grid_dependency_wait();  // the set-up above ran beside the end of the kernel before

    bool timed_out = false;
    GroupedTile t, split = {};
    SchedReader tiles{slots, sched0};
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        const uint32_t bar0 = PAIR ? warp_uniform(map_shared_rank(full0, 0)) : full0;
        const bool issuer = elect_one();
        uint32_t s = 0, phase = 1;
        int issued = 0;
        while (!timed_out && tiles.next(t, tmo, timed_out)) {
            const int mine = ((t.cols + 15) & ~15) / CG;
            const int c0 = t.c0 + rank * mine, f0 = t.f0 + rank * 128;
            const int boxes = (mine + S::kBoxCols - 1) / S::kBoxCols;
            constexpr uint32_t kBox = S::kBoxCols * 128;
            const uint32_t bytes = S::kABytes + boxes * kBox + S::kSaBytes + S::kSbBytes;
            for (int k = t.k0; k < t.k0 + t.klen; k += kMxBK) {
                if (!mbar_wait_warp<false>(empty0 + 8 * s, phase, tmo)) {
                    timed_out = true;
                    break;
                }
                const uint32_t bar = bar0 + 8 * s;
                const uint32_t st = s * S::kStageBytes;
                if (issuer) {
                    auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, int z) {
                        if constexpr (PAIR)
                            tma_load_3d_pair(dst, map, bar, x, y, z);
                        else
                            tma_load_3d(dst, map, bar, x, y, z);
                    };
                    if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, CG * bytes);
                    load(base + st, &tmA, k >> 1, f0, t.e);
#pragma unroll
                    for (int j = 0; j < S::kCols / S::kBoxCols; ++j)
                        if (j < boxes) load(baseB + st + j * kBox, &tmB, k >> 1, c0 + S::kBoxCols * j, 0);
                    // (words; the 8 scales of 256 k are 1024 bytes of 128 rows)
                    load(baseSa + st, &tmSa, k, f0 >> 7, t.e);
                    load(baseSb + st, &tmSb, k, t.srow >> 7, 0);
                }
                __syncwarp();
                ++issued;
                if (++s == S::kStages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        if (timed_out && rank == 0)  // (as in grouped_tc_kernel)
            for (int j = max(0, issued - S::kStages); j < issued; ++j)
                (void)mbar_wait_warp<false>(full0 + 8 * (j % S::kStages), (j / S::kStages) & 1, tmo);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        const uint64_t descA = umma_desc_kmajor_sw128(base), descB = umma_desc_kmajor_sw128(baseB);
        const uint64_t descSa = umma_desc_rows16(baseSa), descSb = umma_desc_rows16(baseSb);
        const uint32_t peer_empty0 = PAIR ? warp_uniform(map_shared_rank(empty0, 1)) : 0;
        const uint32_t peer_acc_full0 = PAIR ? warp_uniform(map_shared_rank(acc_full0, 1)) : 0;
        // float32 accumulator, e2m1 x e2m1, e8m0 scales, M
        constexpr uint32_t kIdesc = 1u << 7 | 1u << 10 | 1u << 23 | static_cast<uint32_t>(FT / 16) << 24;
        const bool issuer = elect_one();
        uint32_t s = 0, phase = 0, turn = 0;  // turn: the scale columns' half
        int unit = 0;
        while (!timed_out && tiles.next(t, tmo, timed_out)) {
            if (rank != 0) continue;
            const uint32_t idesc = kIdesc | static_cast<uint32_t>((t.cols + 15) >> 4) << 18;
            const uint32_t sb_shift = static_cast<uint32_t>((t.srow & 127) >> 5);  // (32 rows of scales a column)
            int k = 0;
            do {
                const int buf = unit & 1, round = unit >> 1;
                const uint32_t acc = tmem + static_cast<uint32_t>(buf * TN);
                const int first = k, end = LONG ? min(t.klen, k + kMxChunk) : t.klen;
                if (round > 0 && !mbar_wait_warp<PAIR>(acc_empty0 + 8 * buf, (round - 1) & 1, tmo)) {
                    timed_out = true;
                    break;
                }
                tc_fence_after_sync();
                for (; k < end; k += kMxBK) {
                    if (!mbar_wait_warp<false>(full0 + 8 * s, phase, tmo)) {
                        timed_out = true;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t off = s * (S::kStageBytes / 16);
                    const uint64_t a = descA + off, b = descB + off, ca = descSa + off, cb = descSb + off;
                    const uint32_t sfa = tmem + S::kScaleCol + turn * S::kScaleCols, sfb = sfa + 8;
                    const int left = t.klen - k;
                    if (issuer) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {  // 128 k: one scale block of each row block
                            if (left > 128 * h) {
                                tmem_cp_32x128b_x4<CG>(sfa + 4 * h, ca + 32 * h);
#pragma unroll
                                for (int j = 0; j < S::kSbBlocks; ++j)
                                    tmem_cp_32x128b_x4<CG>(sfb + 4 * (S::kSbBlocks * h + j), cb + 64 * j + 32 * h);
                            }
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)  // 64 k: scales 0, 1 or 2, 3 of a block
                            if (left > 64 * kk)
                                umma_mxf4<CG>(acc, a + 2 * kk, b + 2 * kk, idesc | (kk & 1 ? 2u << 4 | 2u << 29 : 0u),
                                              sfa + 4 * (kk >> 1), sfb + sb_shift + 4 * S::kSbBlocks * (kk >> 1),
                                              k > first || kk > 0);
                        umma_commit_cg<CG>(empty0 + 8 * s);
                        if constexpr (PAIR) umma_commit_cg<CG>(peer_empty0 + 8 * s);
                    }
                    __syncwarp();
                    turn ^= 1;
                    if (++s == S::kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
                if (timed_out) break;
                if (issuer) {
                    umma_commit_cg<CG>(acc_full0 + 8 * buf);
                    if constexpr (PAIR) umma_commit_cg<CG>(peer_acc_full0 + 8 * buf);
                }
                __syncwarp();
                ++unit;
            } while (LONG && k < t.klen);
        }
        if (timed_out && rank == 0) {
            const int buf = unit & 1, round = unit >> 1;
            if (issuer) umma_commit_cg<CG>(acc_full0 + 8 * buf);
            __syncwarp();
            (void)mbar_wait_warp<false>(acc_full0 + 8 * buf, round & 1, tmo);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ schedule
        GroupCursor cur = p.offsets ? group_begin(p.offsets, p.T) : GroupCursor();
        LastRound last;
        last.set<(PAIR ? TN / 64 : 1)>(mxfp4_tiles<TN>(p), clusters);
        if (!sched_run<TN>(slots, sched0, cluster, clusters, last, tmo,
                           [&](int i, GroupedTile& u) {
                               mxfp4_tile<TN, FT>(p, i, cur, u);
                               if constexpr (SPLIT) split_contraction(u, part, p.ks, kMxBK);
                           }))
            timed_out = true;
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;
        const int half = (warp - 3) >> 2;
        const uint32_t patch = patches + (warp - 3) * kGrPatchBytes;
        const uint32_t acc_empty_lead = PAIR ? warp_uniform(map_shared_rank(acc_empty0, 0)) : acc_empty0;
        if (p.offsets) {
            GroupedTcParams z;  // (the fields that the zeroing reads)
            z.offsets = p.offsets, z.T = p.T, z.E = p.E, z.F = p.F, z.out = p.out, z.ldo = p.ldo;
            const int worker = static_cast<int>(blockIdx.x) * S::kEpiWarps + warp - 3;
            const int workers = static_cast<int>(gridDim.x) * S::kEpiWarps;
            if (p.out_type == 0)
                grouped_zero_rows<float>(z, worker, workers);
            else
                grouped_zero_rows<__half>(z, worker, workers);
        }
        int unit = 0;
        while (!timed_out && tiles.next(t, tmo, timed_out)) {
            const int f = t.f0 + rank * 128 + 32 * q;
            const long long at = static_cast<long long>(t.c0) * p.ldo + f;
            constexpr int kStep = 8 * S::kEpiWarps;  // the warp's columns: 32 of every kStep, from 32 `half` on
            auto wait = [&](uint32_t& acc) {
                const int buf = unit & 1;
                if (!mbar_wait_warp<false>(acc_full0 + 8 * buf, (unit >> 1) & 1, tmo)) return false;
                tc_fence_after_sync();
                acc = tmem + static_cast<uint32_t>(buf * TN) + (static_cast<uint32_t>(32 * q) << 16);
                return true;
            };
            auto release = [&] {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (!PAIR || rank == 0)
                        mbar_arrive(acc_empty0 + 8 * (unit & 1));
                    else
                        mbar_arrive_cluster_relaxed(acc_empty_lead + 8 * (unit & 1));
                }
                __syncwarp();
                ++unit;
            };
            auto put = [&](int c, const auto& v) {
                if constexpr (SPLIT)
                    leave_part(base, c, 32 * q + lane, v);
                else
                    grouped_store<false>(p, patch, at + c * p.ldo, v, t.cols - c, p.F - f);
            };
            uint32_t acc;
            if constexpr (!LONG) {
                if (!wait(acc)) {
                    timed_out = true;
                    break;
                }
                for (int c = 32 * half; c < t.cols; c += kStep) {
                    uint32_t v[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(c), v);
                    tmem_wait_ld();
                    if (SPLIT && t.klen == 0) {  // no MMA wrote the accumulator
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0;
                    }
                    put(c, v);
                }
                release();
            } else {
                float sum[TN / kStep][32];
#pragma unroll
                for (int i = 0; i < TN / kStep; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[i][j] = 0.f;
                for (int k = 0; k < t.klen || k == 0; k += kMxChunk) {
                    if (!wait(acc)) {
                        timed_out = true;
                        break;
                    }
                    if (t.klen > 0) {
#pragma unroll
                        for (int i = 0; i < TN / kStep; ++i) {
                            const int c = 32 * half + kStep * i;
                            if (c < t.cols) {
                                uint32_t v[32];
                                __syncwarp();
                                tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(c), v);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 32; ++j) sum[i][j] += __uint_as_float(v[j]);
                            }
                        }
                    }
                    release();
                }
                if (timed_out) break;
#pragma unroll
                for (int i = 0; i < TN / kStep; ++i) {
                    const int c = 32 * half + kStep * i;
                    if (c < t.cols) put(c, sum[i]);
                }
            }
            if constexpr (SPLIT) split = t;
        }
    }

    if (timed_out) atomicOr(p.status, kGrStatusTimeout);
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();
    if constexpr (SPLIT) {
        cluster_sync_all();
        if (warp >= 3 && split.valid && !timed_out)
            add_parts(p, base, split, part, p.ks, (warp - 3) * 32 + lane, 32 * S::kEpiWarps);
        cluster_sync_all();
    }
    __syncwarp();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_cg<CG>(tmem, S::kTmemCols);
    }
}

}  // namespace gb300
