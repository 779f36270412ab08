// Newton-Schulz products on the fifth-generation tensor cores (tcgen05).
//
// A step on X (m x n, m <= n; where the matrix is taller than wide, what is
// stored is X^T) is three products, each a launch over all matrices:
//
//   gram     A = X X^T            both operands X
//   square   B = b A + c A A      both operands A
//   update   X = a X + B X
//
// Operands are f16, sums float32.  A and B come apart into their diagonals, float32
// vectors d and e, and the rest, O and P, which alone are operands:
//
//   A A = O O + (d_i + d_j) O_ij (i != j),  d_i^2 + (O O)_ii (i = j)
//   X' = (a + e_i) X_ij + (P X)_ij
//
// so that the large elements of a matrix near the identity are not rounded to 11
// bits, and their products cost nothing.  X and A are carried in two
// f16 planes, hi + lo (22 bits); the terms outside of the products use both, the
// products themselves hi alone (PARTS = 1, for bf16 updates) or the three
// products hi hi + hi lo + lo hi (PARTS = 2).  For 1024 x 2048 normal random
// matrices and five steps of the usual polynomial the error of the result's
// norm against 64 bits is 1.8e-3 without the diagonals taken apart and 7e-4 so,
// and with two planes only 4e-7; a matrix of rank 8 and noise 200 times smaller
// is off by 4e-2 if X is one f16 plane, and by 6e-4 so.
//
// Scales.  X is held times 2^13, O and P times 2^12: singular values up to 2
// (the entry refuses polynomials that go beyond) make elements up to 2^14, 2^14
// and 15 * 2^12, below f16's largest.
//
// A and B are symmetric: only tiles that reach the diagonal or lie on its one
// side are computed, and every 32 x 32 block off it is stored twice.
//
// The roles of the warps, the ring and the accumulators are those of
// experts_tc.cuh: load warp, MMA warp, epilogue warps, and persistent CTAs or
// CTA pairs.  The output's rows f lie on the tensor core's rows, its contiguous
// dimension c on the columns, D[f, c] = sum_k P[f, k] Q[c, k] (see the epilogue).  With two planes
// hi hi has an accumulator of its own, the small products another, and both go
// to float32 registers every 512 of the contraction (an instruction cuts
// sums to 24 bits).
//
// Every wait is bounded by `timeout_ns`; on expiry the thread records the
// timeout in the status word and goes to the final barrier.
#pragma once

#include "experts_tc.cuh"

namespace gb300 {

enum OrthoMode { kOrthoGram, kOrthoSquare, kOrthoUpdate };

struct OrthoTcParams {
    int tiles, per;        // output tiles in all, of a matrix
    int ftiles, ctiles;
    int F, C, K, E;        // output F x C (C contiguous), contraction
    const __half* in_hi;   // square: A's planes; update: X's (as the output lies)
    const __half* in_lo;
    __half* out_hi;        // gram: A's planes; square: B's; update: X's next
    __half* out_lo;        // null: not needed
    long long ld_in, s_in, ld_out, s_out;  // elements a row, a matrix
    const float* d_in;     // square: A's diagonals; update: B's (`diag` a matrix, a multiple of 16)
    float* d_out;          // gram: A's diagonals; square: B's
    long long diag;
    int by_column;         // update: e goes by column (else by row)
    float a, b, c;
    void* out;             // the last update's result, of out_type (null: planes)
    long long ldo, so;
    int out_type, align;
    uint32_t idesc;
    unsigned long long timeout_ns;
    unsigned int* status;
};

constexpr int kOrthoChunk = 512;  // contraction in one accumulator, with two planes

template <int TN_, int CG_, int PARTS_>
struct OrthoShape {
    static constexpr int TN = TN_, CG = CG_, PARTS = PARTS_;
    static constexpr int kCols = TN / CG;
    static constexpr int kABytes = 128 * 128, kBBytes = kCols * 128;  // of a part, 64 of the contraction
    static constexpr int kStageBytes = PARTS * (kABytes + kBBytes);
    static constexpr int kEpiWarps = 8;
    static constexpr int kThreads = 32 * (2 + kEpiWarps);
    static constexpr int kPatches = kEpiWarps * kGrPatchBytes;
    static constexpr int kStages = kRing(kStageBytes, kPatches);
    static constexpr int kAccCols = PARTS * TN, kTmemCols = 2 * kAccCols;
    static constexpr int kBars = 2 * kStages + 4;
    static constexpr int kSmem = kStages * kStageBytes + kPatches + 8 * kBars + 16 + 1024;
    static constexpr int kWarpCols = TN / 2;  // an epilogue warp's columns
    static_assert(kSmem <= 227 * 1024 && kStages >= 2 && kCols % 64 == 0 && kTmemCols <= 512, "shape");
};

struct OrthoTile {
    int e, f0, c0;
};

// Tile i: matrix by matrix; of a symmetric output the tiles with a column at or
// below their last feature, feature tile by feature tile (tile f has the first
// (f + 1) FT / TN column tiles, as far as there are any); of the others in
// bands, as the grouped products'.
template <bool SYM, int FT, int TN>
__device__ __forceinline__ OrthoTile ortho_tile(const OrthoTcParams& p, int i) {
    OrthoTile t;
    t.e = i / p.per;
    const int local = i - t.e * p.per;
    int f, c;
    if constexpr (SYM) {
        constexpr int R = FT / TN;
        f = static_cast<int>((sqrtf(8.f * local / R + 1.f) - 1.f) * 0.5f);
        while (R * f * (f + 1) / 2 > local) --f;
        while (R * (f + 1) * (f + 2) / 2 <= local) ++f;
        f = min(f, p.ftiles - 1);
        c = local - R * f * (f + 1) / 2;
    } else {
        tile_place(local, p.ctiles, p.ftiles, f, c);
    }
    t.f0 = f * FT;
    t.c0 = c * TN;
    return t;
}

// ------------------------------------------------------------------ epilogue
//
// A warp takes blocks of 32 rows x 32 columns, a row a lane, so that what a lane
// loads and stores of a plane are 64 neighbouring bytes: two accesses of 32,
// whole sectors, and no way through shared memory.  (With the rows' contiguous
// dimension on the lanes, the products waited for the epilogue: update of 8
// matrices 2048 x 4096 315 us with 2 bytes an access, 188 us with a transposition
// through shared memory.)

struct alignas(32) Half16 {  // 16 f16 values
    uint32_t w[8];
};

// (past the first-level cache, which need not see what the kernel before wrote)
__device__ __forceinline__ Half16 load_half16(const __half* p) {
    Half16 x;
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]), "=r"(x.w[4]), "=r"(x.w[5]), "=r"(x.w[6]), "=r"(x.w[7])
                 : "l"(p));
    return x;
}
__device__ __forceinline__ void store_half16(__half* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// What is carried beside the products at a lane's part of a block: two planes.
template <int MODE>
struct OrthoState {
    Half16 hi[2], lo[2];
    __device__ __forceinline__ void load(const OrthoTcParams& p, int e, int row, int c) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            hi[i] = lo[i] = Half16{};
            if (row < p.F && c + 16 * i < p.C) {
                const long long at = e * p.s_in + row * p.ld_in + c + 16 * i;
                hi[i] = load_half16(p.in_hi + at);
                lo[i] = load_half16(p.in_lo + at);
            }
        }
    }
    __device__ __forceinline__ float value(int j) const {  // (a constant after unrolling)
        const uint32_t h = hi[j / 16].w[j % 16 / 2], l = lo[j / 16].w[j % 16 / 2];
        const __half2 x = *reinterpret_cast<const __half2*>(&h), y = *reinterpret_cast<const __half2*>(&l);
        return j & 1 ? __high2float(x) + __high2float(y) : __low2float(x) + __low2float(y);
    }
};
template <>
struct OrthoState<kOrthoGram> {
    __device__ __forceinline__ void load(const OrthoTcParams&, int, int, int) {}
};

// The diagonals' part of a warp's rows and columns of a tile: the lane's row, and columns 4 lane .. 4 lane + 3.
struct OrthoDiagonal {
    float row = 0.f, column[4] = {};
};

// A block of rows r0 .. and columns c .., from its sums; `first`: its first column among the warp's.
template <int MODE>
__device__ __forceinline__ void ortho_block(const OrthoTcParams& p, uint32_t patch, int e, int r0, int c, int first,
                                            const OrthoState<MODE>& state, const OrthoDiagonal& d, float (&v)[32]) {
    constexpr bool SYM = MODE != kOrthoUpdate;
    const int lane = threadIdx.x & 31, row = r0 + lane;
    const bool diagonal = SYM && r0 == c;
    float* const d_out = p.d_out + e * p.diag;
    const float dr = d.row;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        float dj[4] = {};
        if (MODE == kOrthoSquare || (MODE == kOrthoUpdate && p.by_column)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) dj[i] = __shfl_sync(0xffffffffu, d.column[i], (first + j) / 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float& x = v[j + i];
            const bool on = diagonal && j + i == lane;
            if constexpr (MODE == kOrthoGram) {
                if (on && row < p.F) d_out[row] = x * 0x1p-26f;
                x *= 0x1p-14f;
            } else if constexpr (MODE == kOrthoSquare) {
                if (on && row < p.F) d_out[row] = fmaf(p.c, fmaf(dr, dr, x * 0x1p-24f), p.b * dr);
                const float o = state.value(j + i);
                x = fmaf(p.c, fmaf(dr + dj[i], o, x * 0x1p-12f), p.b * o);
            } else {
                x = fmaf(p.a + (p.by_column ? dj[i] : dr), state.value(j + i), x * 0x1p-12f);
            }
            if (on) x = 0.f;
        }
    }
    if constexpr (MODE == kOrthoUpdate) {
        if (p.out) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= 0x1p-13f;
            const long long at = e * p.so + r0 * p.ldo + c;
            if (p.out_type == 0)
                store_rows(patch, p.align, static_cast<float*>(p.out) + at, p.ldo, v, p.F - r0, p.C - c);
            else if (p.out_type == 1)
                store_rows(patch, p.align, static_cast<__nv_bfloat16*>(p.out) + at, p.ldo, v, p.F - r0, p.C - c);
            else
                store_rows(patch, p.align, static_cast<__half*>(p.out) + at, p.ldo, v, p.F - r0, p.C - c);
            return;
        }
    }
    // hi, then what it leaves.  (Rows of the planes are whole vectors: writing to
    // their ends is harmless.)
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        __half* const plane = part == 0 ? p.out_hi : p.out_lo;
        if (part == 1 && !plane) break;
        __half* const to = plane + e * p.s_out;
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
            v[2 * j] -= __low2float(h);
            v[2 * j + 1] -= __high2float(h);
        }
        if (row < p.F) {
            __half* const at = to + row * p.ld_out + c;
            store_half16(at, w);
            if (c + 16 < p.C) store_half16(at + 16, w + 8);
        }
        if (SYM && !diagonal && row < p.F) {
            // The block's mirror image: rows are columns, a value a lane.
            uint16_t* at = reinterpret_cast<uint16_t*>(to + c * p.ld_out + row);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (c + j < p.C) *at = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
                at += p.ld_out;
            }
        }
    }
}

template <int MODE, bool AMN, bool BMN, int TN, int CG, int PARTS>
__global__ void __launch_bounds__(OrthoShape<TN, CG, PARTS>::kThreads, 1)
    ortho_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const OrthoTcParams p) {
    using S = OrthoShape<TN, CG, PARTS>;
    constexpr bool PAIR = CG == 2, SYM = MODE != kOrthoUpdate;
    constexpr int FT = 128 * CG;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t baseB = base + PARTS * S::kABytes;  // B's parts follow A's in a stage
    const uint32_t patches = base + S::kStages * S::kStageBytes;
    const uint32_t bars = patches + S::kPatches;
    const uint32_t full0 = bars, empty0 = bars + 8 * S::kStages;
    const uint32_t acc_full0 = bars + 16 * S::kStages, acc_empty0 = acc_full0 + 16;
    const uint32_t tmem_slot = bars + 8u * S::kBars;

    const int warp = warp_uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int rank = PAIR ? warp_uniform(static_cast<int>(cluster_ctarank())) : 0;
    const int cluster = static_cast<int>(blockIdx.x) / CG, clusters = static_cast<int>(gridDim.x) / CG;
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
        fence_mbarrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    __syncwarp();
    if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, S::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();  // the peer's barriers are ready
    tc_fence_after_sync();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot) : "memory");
    tmem = warp_uniform(tmem);
    grid_dependency_launch();
    grid_dependency_wait();  // the set-up above ran beside the end of the kernel before

    bool timed_out = false;
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        const uint32_t bar0 = PAIR ? warp_uniform(map_shared_rank(full0, 0)) : full0;
        const bool issuer = elect_one();
        uint32_t s = 0, phase = 1;  // (the first round finds every stage empty)
        int issued = 0;
        for (int i = cluster; i < p.tiles && !timed_out; i += clusters) {
            const OrthoTile t = ortho_tile<SYM, FT, TN>(p, i);
            const int f0 = t.f0 + rank * 128, c0 = t.c0 + rank * S::kCols;
            for (int k = 0; k < p.K; k += kGrBK) {
                if (!mbar_wait_warp<false>(empty0 + 8 * s, phase, tmo)) {
                    timed_out = true;
                    break;
                }
                const uint32_t a = base + s * S::kStageBytes, b = baseB + s * S::kStageBytes;
                if (issuer) {
                    const uint32_t bar = bar0 + 8 * s;
                    if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, CG * S::kStageBytes);
                    auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, int z) {
                        if constexpr (PAIR)
                            tma_load_3d_pair(dst, map, bar, x, y, z);
                        else
                            tma_load_3d(dst, map, bar, x, y, z);
                    };
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        const int z = part * p.E + t.e;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            load(a + part * S::kABytes + j * 64 * 128, &tmA, AMN ? f0 + 64 * j : k, AMN ? k : f0 + 64 * j, z);
#pragma unroll
                        for (int j = 0; j < S::kCols / 64; ++j)
                            load(b + part * S::kBBytes + j * 64 * 128, &tmB, BMN ? c0 + 64 * j : k, BMN ? k : c0 + 64 * j, z);
                    }
                }
                __syncwarp();
                ++issued;
                if (++s == S::kStages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        // (every copy lands before its CTA ends: the MMAs wait for it, and the
        // epilogue for them; after a timeout, the wait below, in the first CTA
        // for the pair)
        if (timed_out && rank == 0)
            for (int j = max(0, issued - S::kStages); j < issued; ++j)
                (void)mbar_wait_warp<false>(full0 + 8 * (j % S::kStages), (j / S::kStages) & 1, tmo);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        if (rank == 0) {  // (the first CTA issues for both)
            const uint64_t descA = AMN ? umma_desc_mnmajor_sw128(base, 64 * 128) : umma_desc_kmajor_sw128(base);
            const uint64_t descB = BMN ? umma_desc_mnmajor_sw128(baseB, 64 * 128) : umma_desc_kmajor_sw128(baseB);
            // 16 k: 32 bytes of each row (K-major), 16 rows of 128 bytes (MN-major); addresses in units of 16
            constexpr uint32_t ka = AMN ? 128 : 2, kb = BMN ? 128 : 2;
            constexpr uint32_t pa = S::kABytes / 16, pb = S::kBBytes / 16;
            const uint32_t peer_empty0 = PAIR ? warp_uniform(map_shared_rank(empty0, 1)) : 0;
            const uint32_t peer_acc_full0 = PAIR ? warp_uniform(map_shared_rank(acc_full0, 1)) : 0;
            const bool issuer = elect_one();
            const uint32_t idesc = p.idesc;
            uint32_t s = 0, phase = 0;
            int unit = 0;  // accumulators filled
            for (int i = cluster; i < p.tiles && !timed_out; i += clusters) {
                for (int k = 0; k < p.K;) {
                    const int buf = unit & 1;
                    const uint32_t acc = tmem + static_cast<uint32_t>(buf * S::kAccCols);
                    const int end = PARTS > 1 ? min(p.K, k + kOrthoChunk) : p.K;
                    if (unit >= 2 && !mbar_wait_warp<PAIR>(acc_empty0 + 8 * buf, ((unit >> 1) - 1) & 1, tmo)) {
                        timed_out = true;
                        break;
                    }
                    tc_fence_after_sync();
                    for (int q = k; q < end; q += kGrBK) {
                        if (!mbar_wait_warp<false>(full0 + 8 * s, phase, tmo)) {
                            timed_out = true;
                            break;
                        }
                        tc_fence_after_sync();
                        const uint32_t off = s * (S::kStageBytes / 16);
                        const uint64_t a = descA + off, b = descB + off;
                        const int left = end - q;
                        if (issuer) {
#pragma unroll
                            for (int kk = 0; kk < kGrBK / 16; ++kk) {
                                if (left > kk * 16) {  // (what lies past the contraction's end is zeros)
                                    const bool add = q > k || kk > 0;
                                    umma_f16<CG>(acc, a + kk * ka, b + kk * kb, idesc, add);
                                    if constexpr (PARTS == 2) {
                                        umma_f16<CG>(acc + TN, a + kk * ka, b + pb + kk * kb, idesc, add);
                                        umma_f16<CG>(acc + TN, a + pa + kk * ka, b + kk * kb, idesc, true);
                                    }
                                }
                            }
                            umma_commit_cg<CG>(empty0 + 8 * s);
                            if constexpr (PAIR) umma_commit_cg<CG>(peer_empty0 + 8 * s);
                        }
                        __syncwarp();
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
                    k = end;
                }
            }
            if (timed_out) {  // the MMAs in flight end before tensor memory is freed
                if (issuer) umma_commit_cg<CG>(acc_full0 + 8 * (unit & 1));
                __syncwarp();
                (void)mbar_wait_warp<false>(acc_full0 + 8 * (unit & 1), (unit >> 1) & 1, tmo);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3, half = (warp - 2) >> 2;
        const uint32_t acc_empty_lead = PAIR ? warp_uniform(map_shared_rank(acc_empty0, 0)) : acc_empty0;
        const uint32_t patch = patches + (warp - 2) * kGrPatchBytes;
        int unit = 0;
        auto wait = [&](uint32_t& acc) {
            const int buf = unit & 1;
            if (!mbar_wait_warp<false>(acc_full0 + 8 * buf, (unit >> 1) & 1, tmo)) return false;
            tc_fence_after_sync();
            acc = tmem + static_cast<uint32_t>(buf * S::kAccCols) + (static_cast<uint32_t>(32 * q) << 16);
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
        for (int i = cluster; i < p.tiles && !timed_out; i += clusters) {
            const OrthoTile t = ortho_tile<SYM, FT, TN>(p, i);
            const int r0 = t.f0 + rank * 128 + 32 * q;  // the warp's first row
            // Blocks of 32 rows x 32 columns: some are not there, or on the diagonal's other side.
            auto wanted = [&](int c) { return r0 < p.F && c < p.C && !(SYM && r0 < c); };
            const int c0 = t.c0 + half * S::kWarpCols;
            // While the MMAs run: the first block's planes, the others' to the second-level cache, the diagonals' parts.
            OrthoState<MODE> next;
            OrthoDiagonal diagonal;
            if (wanted(c0)) next.load(p, t.e, r0 + lane, c0);
            if constexpr (MODE != kOrthoGram) {
                const int row = r0 + lane;
                const float* const d = p.d_in + t.e * p.diag;
                if (row < p.F) {
                    if (MODE == kOrthoSquare || !p.by_column) diagonal.row = __ldcg(d + row);
                    const long long at = t.e * p.s_in + row * p.ld_in + c0;
#pragma unroll
                    for (int j = 32; j < S::kWarpCols; j += 32)
                        if (wanted(c0 + j)) {
                            prefetch_l2(p.in_hi + at + j);
                            prefetch_l2(p.in_lo + at + j);
                        }
                }
                if ((MODE == kOrthoSquare || p.by_column) && 4 * lane < S::kWarpCols && c0 + 4 * lane < p.C) {
                    const float4 x = __ldcg(reinterpret_cast<const float4*>(d + c0) + lane);
                    diagonal.column[0] = x.x, diagonal.column[1] = x.y, diagonal.column[2] = x.z, diagonal.column[3] = x.w;
                }
            }
            auto block = [&](int j, float (&v)[32]) {
                const OrthoState<MODE> state = next;
                if (32 * (j + 1) < S::kWarpCols && wanted(c0 + 32 * (j + 1))) next.load(p, t.e, r0 + lane, c0 + 32 * (j + 1));
                if (wanted(c0 + 32 * j)) ortho_block<MODE>(p, patch, t.e, r0, c0 + 32 * j, 32 * j, state, diagonal, v);
            };
            uint32_t acc;
            if constexpr (PARTS == 1) {
                if (!wait(acc)) {
                    timed_out = true;
                    break;
                }
#pragma unroll 1
                for (int j = 0; j < S::kWarpCols / 32; ++j) {
                    uint32_t r[32];
                    float v[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(half * S::kWarpCols + 32 * j), r);
                    tmem_wait_ld();
#pragma unroll
                    for (int u = 0; u < 32; ++u) v[u] = __uint_as_float(r[u]);
                    block(j, v);
                }
                release();
            } else {
                float sum[S::kWarpCols / 32][32];
#pragma unroll
                for (int j = 0; j < S::kWarpCols / 32; ++j)
#pragma unroll
                    for (int u = 0; u < 32; ++u) sum[j][u] = 0.f;
                for (int k = 0; k < p.K; k += kOrthoChunk) {
                    if (!wait(acc)) {
                        timed_out = true;
                        break;
                    }
#pragma unroll
                    for (int j = 0; j < S::kWarpCols / 32; ++j) {
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
                            const uint32_t c = static_cast<uint32_t>(half * S::kWarpCols + 32 * j + h);
                            uint32_t big[16], small[16];
                            __syncwarp();
                            tmem_ld_32x32b_x16(acc + TN + c, small);
                            tmem_ld_32x32b_x16(acc + c, big);
                            tmem_wait_ld();
#pragma unroll
                            for (int u = 0; u < 16; ++u)
                                sum[j][h + u] += __uint_as_float(big[u]) + __uint_as_float(small[u]);
                        }
                    }
                    release();
                }
                if (timed_out) break;
#pragma unroll
                for (int j = 0; j < S::kWarpCols / 32; ++j) block(j, sum[j]);
            }
        }
    }

    if (timed_out) atomicOr(p.status, kGrStatusTimeout);
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();  // nothing of the peer's is under way in this CTA's memory
    __syncwarp();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_cg<CG>(tmem, S::kTmemCols);
    }
}

}  // namespace gb300
