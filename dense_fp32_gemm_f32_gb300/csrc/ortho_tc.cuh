// Newton-Schulz products on the fifth-generation tensor cores (tcgen05).
//
// A step on X (m x n, m <= n; where the matrix is taller than wide, what is
// stored is X^T) is three products:
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
// products themselves the three hi hi + hi lo + lo hi (PARTS = 2) or, for bf16
// updates whose caller asks for it, hi alone (PARTS = 1).  For 1024 x 2048 normal random
// matrices and five steps of the usual polynomial the error of the result's
// norm against 64 bits is 1.8e-3 without the diagonals taken apart and 7e-4 so,
// and with products of two planes 4e-7; a matrix of rank 8 and noise 200 times smaller
// is off by 4e-2 if X is one f16 plane, and by 6e-4 so.  The error of one plane
// is half of bf16's rounding of the result, but grows with the steps and with what the polynomial raises:
// it is the caller's choice.
//
// Scales.  X is held times 2^13, O and P times 2^12: singular values up to 2
// (the entry refuses polynomials that go beyond) make elements up to 2^14, 2^14
// and 15 * 2^12, below f16's largest.
//
// A and B are symmetric: where there are more tiles than the GPU's pairs of CTAs,
// only those that reach the diagonal or lie on its one side are computed, and every
// 32 x 32 block off it is stored twice.  (Where there are fewer, the second
// store, 2 bytes a lane, is the longer way: 129 x 129 bf16 79 us with it.)
//
// All steps are one launch.  Its CTA pairs are resident together (a cooperative
// launch) and take the output tiles of all products in one order,
// every P-th each; a tile waits until the row panels that it reads are there:
//
//   gram tile (i, j)       rows i and j of X           (panels of FT rows)
//   square tile (i, j)     rows i and j of A
//   update tile (r, c)     rows r of B (taller than wide: c), and so all of A and X
//
// A counter a panel holds the CTAs that have finished a tile with rows in it,
// over all steps.  Tiles come in an order in which every tile waits for
// earlier ones alone, so the first unfinished one can always proceed.  A buffer
// is written again only by tiles that wait, through others, for all that read it
// before (X alternates between two).  Products of several matrices then follow one another without a
// gap, and those of one matrix with gaps of about a tile.
//
// The roles of the warps, the ring and the accumulators are those of
// experts_tc.cuh: load warp, MMA warp, epilogue warps.  The output's rows f lie on
// the tensor core's rows, its contiguous dimension c on the columns, D[f, c] =
// sum_k P[f, k] Q[c, k] (see the epilogue).  With two planes
// hi hi has an accumulator of its own, the small products another, and both go
// to float32 registers every 512 of the contraction (an instruction cuts
// sums to 24 bits).
//
// Measured on GB300, five steps, of bf16 (of float32 the same but for 2 to 4 %): 8 matrices 2048 x 4096 5.2 to 5.35 ms,
// 1.8 with products of one plane (with 5 / 8 of the symmetric products' flops 1.5 PFLOP/s in either; the GPU runs at its
// power limit, 1.6 GHz, at which the tensor pipe would need 1.5 of the 1.8 ms; preparation 95 us); 1024 x 1024 138 us and
// 100, 512 x 512 101 and 78, bound by latency: of the 8000 to 9000 cycles of a tile of 128 columns on the way from one product to the next 1100 are the
// first copy's, 1000 to 2400 the products', 3300 the epilogue's and 1900 the counters'.
//
// (ptxas: 216 and 248 bytes of spills with tiles of 128 columns and two planes, whose 18 warps have 96 registers a thread; 10 warps of
// 168 are slower all the same, see kEpiWarps.)
//
// Every wait is bounded by `timeout_ns`; on expiry the thread records the
// timeout in the status word and goes to the final barrier.
#pragma once

#include "experts_tc.cuh"
#include "ortho_load.cuh"

namespace gb300 {

enum OrthoPhase { kOrthoGram, kOrthoSquare, kOrthoUpdate };

// Matrices in two f16 planes, E in each.
struct OrthoPlanes {
    __half *hi, *lo;       // (lo of B: of two planes alone)
    long long ld, matrix;  // elements a row, a matrix
};

struct OrthoTcParams {
    int E, m, rows, cols;     // X as stored: rows x cols, m the shorter
    int steps, items;         // output tiles in all
    int sym_tiles, up_tiles;  // of a matrix: gram or square, update
    int mirror;               // gram and square: tiles on one side of the diagonal alone, stored twice
    OrthoPlanes x[2], a, p;   // X (by turns), A and B less their diagonals
    float *d, *e;             // the diagonals of A and B, `diag` (a multiple of 16) a matrix
    long long diag;
    int* done;                // counters: 3 kinds (X, A, B) x E x panels, zero at the start
    int panels;
    float c1, c3, c5;         // the polynomial
    const int* shift;         // of each matrix: X is held times this power of two besides, less `growth` a step (ortho_load.cuh)
    int growth;
    void* out;
    long long ldo, so;
    int out_type, align;
    unsigned long long timeout_ns;
    unsigned int* status;
};

constexpr int kOrthoChunk = 512;  // contraction in one accumulator, with two planes
constexpr int kOrthoSlots = 4;    // tiles that the load warp tells the epilogue warps about ahead

template <int TN_, int PARTS_>
struct OrthoShape {
    static constexpr int TN = TN_, PARTS = PARTS_;
    static constexpr int FT = 256, R = FT / TN;  // a tile's rows; column tiles of a panel
    static constexpr int kCols = TN / 2;         // of a CTA
    // of a part, 64 of the contraction (boxes of 64 rows or columns, of which the narrowest tile takes the first 32)
    static constexpr int kBoxes = (kCols + 63) / 64, kABytes = 128 * 128, kBBytes = kBoxes * 64 * 128;
    static constexpr int kStageBytes = PARTS * (kABytes + kBBytes);
    // Measured, 8 and 16 warps (168 and 96 registers a thread): tiles of 256 columns, 8 x 2048 x 4096 bf16 1740 and 1880
    // us; of 128 columns and two planes, 4 x 2048 x 2048 float32 1470 and 1415 us.
    static constexpr int kEpiWarps = TN == 128 ? 16 : 8;
    static constexpr int kThreads = 32 * (2 + kEpiWarps);
    // (the widest tile has a seventh stage instead of patches for results off the 16-byte grid)
    static constexpr bool kPatched = !(TN == 256 && PARTS == 1);
    static constexpr int kPatches = kPatched ? kEpiWarps * kGrPatchBytes : 0;
    static constexpr int kStages = kRing(kStageBytes, kPatches);
    static constexpr int kAccCols = PARTS * TN, kTmemCols = 2 * kAccCols;
    static constexpr int kBars = 2 * kStages + 4 + 2 * kOrthoSlots;
    static constexpr int kSmem = kStages * kStageBytes + kPatches + 8 * kBars + 32 + 1024;
    static constexpr int kWarpCols = TN / (kEpiWarps / 4);  // an epilogue warp's columns
    static constexpr int kDone = 2;                         // what a tile's CTAs add to a panel's counter
    static_assert(kSmem <= 227 * 1024 && kStages >= 2 && kCols % 32 == 0 && kWarpCols % 32 == 0 && kTmemCols <= 512 && FT % TN == 0, "shape");
};

__device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }

// Adds one to a word of shared memory; what it was.  Ordered as a release and an acquire.
__device__ __forceinline__ uint32_t count_shared(uint32_t addr) {
    uint32_t was;
    asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(was) : "r"(addr) : "memory");
    return was;
}

struct OrthoTile {
    int step, phase, e, f0, c0;
    int need0, need1;  // panels that it reads
};

// Item i: step by step, product by product, matrix by matrix.  A gram tile's
// panels are those that the update before it finishes first (row by row, up to
// the diagonal), a square tile's order finishes panel after panel of B for the
// update (column panel by column panel, from the diagonal down).
template <typename S, bool TALL>
__device__ __forceinline__ OrthoTile ortho_tile(const OrthoTcParams& p, int i) {
    OrthoTile t;
    const int sym = p.E * p.sym_tiles, all = 2 * sym + p.E * p.up_tiles;
    t.step = i / all;
    int local = i - t.step * all;
    if (local < 2 * sym) {
        t.phase = local < sym ? kOrthoGram : kOrthoSquare;
        if (t.phase == kOrthoSquare) local -= sym;
        t.e = local / p.sym_tiles;
        local -= t.e * p.sym_tiles;
        const int ft = div_up(p.m, S::FT), ct = div_up(p.m, S::TN);
        int f = 0, c;
        if (!p.mirror) {
            f = local / ct;
            c = local - f * ct;
        } else if (t.phase == kOrthoGram) {
            while (true) {
                const int n = min(ct, (f + 1) * S::R);
                if (local < n) break;
                local -= n;
                ++f;
            }
            c = local;
        } else {
            int q = 0, width;
            while (true) {
                width = min(S::R, ct - q * S::R);
                const int n = (ft - q) * width;
                if (local < n) break;
                local -= n;
                ++q;
            }
            f = q + local / width;
            c = q * S::R + local % width;
        }
        t.f0 = f * S::FT;
        t.c0 = c * S::TN;
        t.need0 = f;
        t.need1 = c / S::R;
    } else {
        t.phase = kOrthoUpdate;
        local -= 2 * sym;
        t.e = local / p.up_tiles;
        local -= t.e * p.up_tiles;
        int f, c;
        if constexpr (TALL) {
            const int ft = div_up(p.rows, S::FT);
            c = local / ft;
            f = local - c * ft;
            t.need0 = t.need1 = c / S::R;
        } else {
            const int ct = div_up(p.cols, S::TN);
            f = local / ct;
            c = local - f * ct;
            t.need0 = t.need1 = f;
        }
        t.f0 = f * S::FT;
        t.c0 = c * S::TN;
    }
    return t;
}

// The counter that panel `q` of what tile t reads has reached when it is there.
template <typename S, bool TALL>
__device__ __forceinline__ int ortho_needed(const OrthoTcParams& p, const OrthoTile& t, int q) {
    const int ft = div_up(p.m, S::FT), ct = div_up(p.m, S::TN);
    const int width = min(S::R, ct - q * S::R);  // column tiles of the panel
    if (t.phase == kOrthoGram)  // X, of the step before
        return t.step * S::kDone * (TALL ? div_up(p.rows, S::FT) * width : div_up(p.cols, S::TN));
    return (t.step + 1) * S::kDone * (p.mirror ? min(ct, (q + 1) * S::R) + (ft - 1 - q) * width : ct);
}

// Whole warp: waits until the panels that tile t reads are there.  Without
// mirrored tiles a gram tile waits for all of X (at most 32 panels; the host sees
// to it): it overwrites rows of A that square tiles of other panels have read.
template <typename S, bool TALL>
__device__ __forceinline__ bool ortho_wait(const OrthoTcParams& p, const OrthoTile& t) {
    const int lane = threadIdx.x & 31;
    const bool all = !p.mirror && t.phase == kOrthoGram;
    const int q = all ? min(lane, p.panels - 1) : lane == 0 ? t.need0 : t.need1;
    const int* counter = p.done + (static_cast<long long>(t.phase) * p.E + t.e) * p.panels + q;
    const int needed = ortho_needed<S, TALL>(p, t, q);
    auto ready = [&] { return __all_sync(0xffffffffu, (lane > 1 && !all) || load_acquire_gpu(counter) >= needed) != 0; };
    uint64_t t0 = 0;
    while (!ready()) {
        const uint64_t now = global_timer_ns();
        if (t0 == 0)
            t0 = now;
        else if (__any_sync(0xffffffffu, now - t0 > p.timeout_ns))
            return false;
    }
    __syncwarp();  // (what two lanes have acquired, all may read)
    return true;
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

// (past the first-level cache: other SMs write what is read here)
__device__ __forceinline__ Half16 load_half16(const __half* p) {
    Half16 x;
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]), "=r"(x.w[4]), "=r"(x.w[5]), "=r"(x.w[6]), "=r"(x.w[7])
                 : "l"(p)
                 : "memory");
    return x;
}
__device__ __forceinline__ void store_half16(__half* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// What is carried beside the products at a lane's part of a block: two planes.
struct OrthoState {
    Half16 hi[2], lo[2];
    __device__ __forceinline__ void load(const __half* h, const __half* l, bool first, bool second) {
        hi[0] = hi[1] = lo[0] = lo[1] = Half16{};
        if (first) hi[0] = load_half16(h), lo[0] = load_half16(l);
        if (second) hi[1] = load_half16(h + 16), lo[1] = load_half16(l + 16);
    }
    __device__ __forceinline__ float value(int j) const {  // (j: a constant after unrolling)
        const uint32_t h = hi[j / 16].w[j % 16 / 2], l = lo[j / 16].w[j % 16 / 2];
        const __half2 x = *reinterpret_cast<const __half2*>(&h), y = *reinterpret_cast<const __half2*>(&l);
        return j & 1 ? __high2float(x) + __high2float(y) : __low2float(x) + __low2float(y);
    }
};

// What the power of two that a matrix's X is held times (see ortho_load.cuh) makes of the polynomial in this step.
struct OrthoPowers {
    float c3, c5;     // of a square
    float step, out;  // of an update: 2^(q' - q), and what X is divided by in the end
    __device__ __forceinline__ OrthoPowers(const OrthoTcParams& p, const OrthoTile& t, int shift) {
        const int q = max(0, shift - t.step * p.growth), next = max(0, q - p.growth);
        c3 = p.c3 * power_of_two(-2 * q);
        c5 = p.c5 * power_of_two(-4 * q);
        step = power_of_two(next - q);
        out = 0x1p-13f * power_of_two(-next);
    }
};

// The diagonals' part of a warp's rows and columns of a tile: the lane's row, and columns 4 lane .. 4 lane + 3.
struct OrthoDiagonal {
    float row, column[4];
};

// A block of the result in its own type, a row a lane; rows and columns that there are.
template <typename S, typename T>
__device__ __forceinline__ void ortho_result(const OrthoTcParams& p, uint32_t patch, long long at, const float (&v)[32],
                                             int rows, int cols) {
    T* const o = static_cast<T*>(p.out) + at;
    const int lane = threadIdx.x & 31;
    if (p.align == 16 && cols >= 32) {
        if (lane < rows) {
            uint4* to = reinterpret_cast<uint4*>(o + lane * p.ldo);
#pragma unroll
            for (int j = 0; j < 32; j += 16 / static_cast<int>(sizeof(T))) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (sizeof(T) == 4)
                        w[i] = __float_as_uint(v[j + i]);
                    else
                        w[i] = pair_from_f32<T>(v[j + 2 * i], v[j + 2 * i + 1]);
                }
                *to++ = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    } else if constexpr (S::kPatched) {
        store_rows(patch, p.align, o, p.ldo, v, rows, cols);
    } else if (lane < rows) {
        T* to = o + lane * p.ldo;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < cols) to[j] = from_f32<T>(v[j]);
    }
}

// A block of rows r0 .. and columns c .. of tile t, from its sums; `first`: its first column among the warp's.
template <typename S, bool TALL, int PHASE>
__device__ __forceinline__ void ortho_block(const OrthoTcParams& p, uint32_t patch, const OrthoTile& t, int r0, int c,
                                            int first, const OrthoState& state, const OrthoDiagonal& d, const OrthoPowers& w,
                                            float (&v)[32]) {
    constexpr bool SYM = PHASE != kOrthoUpdate;
    const int lane = threadIdx.x & 31, row = r0 + lane;
    const int F = SYM ? p.m : p.rows, C = SYM ? p.m : p.cols;
    const bool diagonal = SYM && r0 == c;
    float* const d_out = (PHASE == kOrthoGram ? p.d : p.e) + t.e * p.diag;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        float dj[4] = {};
        if (PHASE == kOrthoSquare || (PHASE == kOrthoUpdate && TALL)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) dj[i] = __shfl_sync(0xffffffffu, d.column[i], (first + j) / 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float& x = v[j + i];
            const bool on = diagonal && j + i == lane;
            if constexpr (PHASE == kOrthoGram) {
                if (on && row < F) d_out[row] = x * 0x1p-26f;
                x *= 0x1p-14f;
            } else if constexpr (PHASE == kOrthoSquare) {
                if (on && row < F) d_out[row] = fmaf(w.c5, fmaf(d.row, d.row, x * 0x1p-24f), w.c3 * d.row);
                const float o = state.value(j + i);
                x = fmaf(w.c5, fmaf(d.row + dj[i], o, x * 0x1p-12f), w.c3 * o);
            } else {
                x = w.step * fmaf(p.c1 + (TALL ? dj[i] : d.row), state.value(j + i), x * 0x1p-12f);
            }
            if (on) x = 0.f;
        }
    }
    if constexpr (PHASE == kOrthoUpdate) {
        if (t.step + 1 == p.steps) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= w.out;
            const long long at = t.e * p.so + r0 * p.ldo + c;
            if constexpr (S::PARTS == 1) {
                ortho_result<S, __nv_bfloat16>(p, patch, at, v, F - r0, C - c);
            } else {
                if (p.out_type == 0)
                    ortho_result<S, float>(p, patch, at, v, F - r0, C - c);
                else if (p.out_type == 1)
                    ortho_result<S, __nv_bfloat16>(p, patch, at, v, F - r0, C - c);
                else
                    ortho_result<S, __half>(p, patch, at, v, F - r0, C - c);
            }
            return;
        }
    }
    // hi, then what it leaves.  (Rows of the planes are whole vectors: writing to
    // their ends is harmless.)
    const OrthoPlanes& to = PHASE == kOrthoGram ? p.a : PHASE == kOrthoSquare ? p.p : p.x[(t.step & 1) ^ 1];
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        if (part == 1 && PHASE == kOrthoSquare && S::PARTS == 1) break;  // (products take B's hi alone)
        __half* const plane = (part == 0 ? to.hi : to.lo) + t.e * to.matrix;
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
            v[2 * j] -= __low2float(h);
            v[2 * j + 1] -= __high2float(h);
        }
        if (row < F) {
            __half* const at = plane + row * to.ld + c;
            store_half16(at, w);
            if (c + 16 < C) store_half16(at + 16, w + 8);
        }
        if (SYM && p.mirror && !diagonal && row < F) {
            // The block's mirror image: rows are columns, a value a lane.
            uint16_t* at = reinterpret_cast<uint16_t*>(plane + c * to.ld + row);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (c + j < C) *at = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
                at += to.ld;
            }
        }
    }
}

template <int TN, int PARTS, bool TALL>
__global__ void __launch_bounds__(OrthoShape<TN, PARTS>::kThreads, 1)
    ortho_tc_kernel(const __grid_constant__ CUtensorMap tm_x0, const __grid_constant__ CUtensorMap tm_x1,
                    const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_p,
                    const OrthoTcParams p) {
    using S = OrthoShape<TN, PARTS>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t baseB = base + PARTS * S::kABytes;  // the second operand's parts follow the first's in a stage
    const uint32_t patches = base + S::kStages * S::kStageBytes;
    const uint32_t bars = patches + S::kPatches;
    const uint32_t full0 = bars, empty0 = bars + 8 * S::kStages;
    const uint32_t acc_full0 = bars + 16 * S::kStages, acc_empty0 = acc_full0 + 16;
    const uint32_t there0 = acc_empty0 + 16, seen0 = there0 + 8 * kOrthoSlots;  // what a tile reads is there; has been read
    const uint32_t tmem_slot = bars + 8u * S::kBars, finished = tmem_slot + 4;  // finished: warps, by slot

    const int warp = warp_uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int rank = warp_uniform(static_cast<int>(cluster_ctarank()));
    const int cluster = static_cast<int>(blockIdx.x) / 2, clusters = static_cast<int>(gridDim.x) / 2;
    const unsigned long long tmo = p.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full0 + 8 * b, 1);
            mbar_init(acc_empty0 + 8 * b, 2 * S::kEpiWarps);
        }
        for (int j = 0; j < kOrthoSlots; ++j) {
            mbar_init(there0 + 8 * j, 1);
            mbar_init(seen0 + 8 * j, S::kEpiWarps);
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(finished + 4 * j), "r"(0) : "memory");
        }
        fence_mbarrier_init();
        prefetch_tensormap(&tm_x0);
        prefetch_tensormap(&tm_x1);
        prefetch_tensormap(&tm_a);
        prefetch_tensormap(&tm_p);
    }
    __syncwarp();
    if (warp == 1) tmem_alloc_cg<2>(tmem_slot, S::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();  // the peer's barriers are ready
    tc_fence_after_sync();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot) : "memory");
    tmem = warp_uniform(tmem);

    auto contraction = [&](int phase) { return phase == kOrthoGram ? (TALL ? p.rows : p.cols) : p.m; };
    bool timed_out = false;
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        const uint32_t bar0 = warp_uniform(map_shared_rank(full0, 0));
        const bool issuer = elect_one();
        uint32_t s = 0, phase = 1;  // (the first round finds every stage empty)
        int issued = 0, n = 0;
        for (int i = cluster; i < p.items && !timed_out; i += clusters, ++n) {
            const OrthoTile t = ortho_tile<S, TALL>(p, i);
            const int slot = n % kOrthoSlots, round = n / kOrthoSlots;
            if ((round > 0 && !mbar_wait_warp<false>(seen0 + 8 * slot, (round - 1) & 1, 3 * tmo)) ||
                !ortho_wait<S, TALL>(p, t)) {
                timed_out = true;
                break;
            }
            if (issuer) mbar_arrive(there0 + 8 * slot);
            __syncwarp();
            fence_proxy_async_global();  // (the copies read what other SMs stored)
            const CUtensorMap* const x = t.step & 1 ? &tm_x1 : &tm_x0;
            const CUtensorMap* const first = t.phase == kOrthoGram ? x : t.phase == kOrthoSquare ? &tm_a : TALL ? x : &tm_p;
            const CUtensorMap* const second = t.phase == kOrthoGram ? x : t.phase == kOrthoSquare ? &tm_a : TALL ? &tm_p : x;
            const bool first_mn = TALL && t.phase == kOrthoGram;
            const bool second_mn = TALL ? t.phase == kOrthoGram : t.phase == kOrthoUpdate;
            const int f0 = t.f0 + rank * 128, c0 = t.c0 + rank * S::kCols, K = contraction(t.phase);
            for (int k = 0; k < K; k += kGrBK) {
                if (!mbar_wait_warp<false>(empty0 + 8 * s, phase, tmo)) {
                    timed_out = true;
                    break;
                }
                const uint32_t a = base + s * S::kStageBytes, b = baseB + s * S::kStageBytes;
                if (issuer) {
                    const uint32_t bar = bar0 + 8 * s;
                    if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, 2 * S::kStageBytes);
                    auto load = [&](uint32_t dst, const CUtensorMap* map, bool mn, int at, int z) {
                        const int x0 = mn ? at : k, y0 = mn ? k : at;
                        tma_load_3d_pair(dst, map, bar, x0, y0, z);
                    };
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        const int z = part * p.E + t.e;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            load(a + part * S::kABytes + j * 64 * 128, first, first_mn, f0 + 64 * j, z);
#pragma unroll
                        for (int j = 0; j < S::kBoxes; ++j)
                            load(b + part * S::kBBytes + j * 64 * 128, second, second_mn, c0 + 64 * j, z);
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
            constexpr uint32_t pa = S::kABytes / 16, pb = S::kBBytes / 16;
            const uint32_t peer_empty0 = warp_uniform(map_shared_rank(empty0, 1));
            const uint32_t peer_acc_full0 = warp_uniform(map_shared_rank(acc_full0, 1));
            const bool issuer = elect_one();
            uint32_t s = 0, phase = 0;
            int unit = 0;  // accumulators filled
            for (int i = cluster; i < p.items && !timed_out; i += clusters) {
                const int of = ortho_tile<S, TALL>(p, i).phase, K = contraction(of);
                const bool a_mn = TALL && of == kOrthoGram, b_mn = TALL ? of == kOrthoGram : of == kOrthoUpdate;
                const uint64_t descA = a_mn ? umma_desc_mnmajor_sw128(base, 64 * 128) : umma_desc_kmajor_sw128(base);
                const uint64_t descB = b_mn ? umma_desc_mnmajor_sw128(baseB, 64 * 128) : umma_desc_kmajor_sw128(baseB);
                // 16 k: 32 bytes of each row (K-major), 16 rows of 128 bytes (MN-major); addresses in units of 16
                const uint32_t ka = a_mn ? 128 : 2, kb = b_mn ? 128 : 2;
                const uint32_t idesc = 1u << 4 | (a_mn ? 1u << 15 : 0) | (b_mn ? 1u << 16 : 0) |
                                       static_cast<uint32_t>(TN / 8) << 17 | static_cast<uint32_t>(S::FT / 16) << 24;
                for (int k = 0; k < K;) {
                    const int buf = unit & 1;
                    const uint32_t acc = tmem + static_cast<uint32_t>(buf * S::kAccCols);
                    const int end = PARTS > 1 ? min(K, k + kOrthoChunk) : K;
                    if (unit >= 2 && !mbar_wait_warp<true>(acc_empty0 + 8 * buf, ((unit >> 1) - 1) & 1, tmo)) {
                        timed_out = true;
                        break;
                    }
                    tc_fence_after_sync();
                    for (int q = k; q < end; q += kGrBK) {
                        // (the load warp waits for what it reads up to the limit, and then for the stage)
                        if (!mbar_wait_warp<false>(full0 + 8 * s, phase, 2 * tmo)) {
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
                                    umma_f16<2>(acc, a + kk * ka, b + kk * kb, idesc, add);
                                    if constexpr (PARTS == 2) {
                                        umma_f16<2>(acc + TN, a + kk * ka, b + pb + kk * kb, idesc, add);
                                        umma_f16<2>(acc + TN, a + pa + kk * ka, b + kk * kb, idesc, true);
                                    }
                                }
                            }
                            umma_commit_cg<2>(empty0 + 8 * s);
                            umma_commit_cg<2>(peer_empty0 + 8 * s);
                        }
                        __syncwarp();
                        if (++s == S::kStages) {
                            s = 0;
                            phase ^= 1;
                        }
                    }
                    if (timed_out) break;
                    if (issuer) {
                        umma_commit_cg<2>(acc_full0 + 8 * buf);
                        umma_commit_cg<2>(peer_acc_full0 + 8 * buf);
                    }
                    __syncwarp();
                    ++unit;
                    k = end;
                }
            }
            if (timed_out) {  // the MMAs in flight end before tensor memory is freed
                if (issuer) umma_commit_cg<2>(acc_full0 + 8 * (unit & 1));
                __syncwarp();
                (void)mbar_wait_warp<false>(acc_full0 + 8 * (unit & 1), (unit >> 1) & 1, tmo);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3, share = (warp - 2) >> 2;
        const uint32_t acc_empty_lead = warp_uniform(map_shared_rank(acc_empty0, 0));
        const uint32_t patch = patches + (warp - 2) * kGrPatchBytes;
        int unit = 0, n = 0;
        auto wait = [&](uint32_t& acc) {
            const int buf = unit & 1;
            if (!mbar_wait_warp<false>(acc_full0 + 8 * buf, (unit >> 1) & 1, 4 * tmo)) return false;
            tc_fence_after_sync();
            acc = tmem + static_cast<uint32_t>(buf * S::kAccCols) + (static_cast<uint32_t>(32 * q) << 16);
            return true;
        };
        auto release = [&] {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (rank == 0)
                    mbar_arrive(acc_empty0 + 8 * (unit & 1));
                else
                    mbar_arrive_cluster_relaxed(acc_empty_lead + 8 * (unit & 1));
            }
            __syncwarp();
            ++unit;
        };
        // A tile of product PHASE; false on a timeout.
        auto tile = [&](const OrthoTile& t, auto which) -> bool {
            constexpr int PHASE = decltype(which)::value;
            constexpr bool SYM = PHASE != kOrthoUpdate;
            const int F = SYM ? p.m : p.rows, C = SYM ? p.m : p.cols, K = contraction(PHASE);
            const int r0 = t.f0 + rank * 128 + 32 * q, c0 = t.c0 + share * S::kWarpCols;  // the warp's first row and column
            // Blocks of 32 rows x 32 columns: some are not there, or on the diagonal's other side.
            auto wanted = [&](int c) { return r0 < F && c < C && !(SYM && p.mirror && r0 < c); };
            // While the MMAs run: the first block's planes, the diagonals' parts.
            OrthoState next = {};
            OrthoDiagonal diagonal = {};
            const __half *hi = nullptr, *lo = nullptr;
            const bool mine = r0 + lane < F;
            const OrthoPowers powers(p, t, __ldg(p.shift + t.e));
            if (!mbar_wait_warp<false>(there0 + 8 * (n % kOrthoSlots), (n / kOrthoSlots) & 1, 4 * tmo)) return false;
            if constexpr (PHASE != kOrthoGram) {
                const OrthoPlanes& from = PHASE == kOrthoSquare ? p.a : p.x[t.step & 1];
                const long long at = t.e * from.matrix + (r0 + lane) * from.ld + c0;
                hi = from.hi + at;
                lo = from.lo + at;
                const float* const d = (PHASE == kOrthoSquare ? p.d : p.e) + t.e * p.diag;
                if (wanted(c0)) next.load(hi, lo, mine, mine && c0 + 16 < C);
                if (mine && (PHASE == kOrthoSquare || !TALL)) diagonal.row = __ldcg(d + r0 + lane);
                if ((PHASE == kOrthoSquare || TALL) && 4 * lane < S::kWarpCols && c0 + 4 * lane < C) {
                    const float4 x = __ldcg(reinterpret_cast<const float4*>(d + c0) + lane);
                    diagonal.column[0] = x.x, diagonal.column[1] = x.y, diagonal.column[2] = x.z, diagonal.column[3] = x.w;
                }
            }
            auto block = [&](int j, float (&v)[32]) {
                const int c = c0 + 32 * j;
                if (wanted(c)) ortho_block<S, TALL, PHASE>(p, patch, t, r0, c, 32 * j, next, diagonal, powers, v);
                if (PHASE != kOrthoGram && 32 * (j + 1) < S::kWarpCols && wanted(c + 32))
                    next.load(hi + 32 * (j + 1), lo + 32 * (j + 1), mine, mine && c + 48 < C);
            };
            uint32_t acc;
            if constexpr (PARTS == 1) {
                if (!wait(acc)) return false;
#pragma unroll 1
                for (int j = 0; j < S::kWarpCols / 32; ++j) {
                    uint32_t r[32];
                    float v[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(share * S::kWarpCols + 32 * j), r);
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
                for (int k = 0; k < K; k += kOrthoChunk) {
                    if (!wait(acc)) return false;
#pragma unroll
                    for (int j = 0; j < S::kWarpCols / 32; ++j) {
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
                            const uint32_t c = static_cast<uint32_t>(share * S::kWarpCols + 32 * j + h);
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
#pragma unroll
                for (int j = 0; j < S::kWarpCols / 32; ++j) block(j, sum[j]);
            }
            // The CTA's last warp tells those that wait for the tile's rows and for those of its mirror image.
            fence_proxy_async_global();
            __syncwarp();
            if (lane == 0) {
                const int slot = n % kOrthoSlots;
                if (count_shared(finished + 4 * slot) % S::kEpiWarps == S::kEpiWarps - 1 &&
                    (PHASE != kOrthoUpdate || t.step + 1 < p.steps)) {
                    // kinds: gram finishes A (1), square B (2), update X (0)
                    constexpr int kind = PHASE == kOrthoUpdate ? 0 : PHASE + 1;
                    int* const counter = p.done + (static_cast<long long>(kind) * p.E + t.e) * p.panels;
                    add_release_gpu(counter + t.need0, 1);
                    if (SYM && p.mirror && t.need1 != t.need0) add_release_gpu(counter + t.need1, 1);
                }
                mbar_arrive(seen0 + 8 * slot);  // (after the count: the slot is used again when all have arrived)
            }
            __syncwarp();
            ++n;
            return true;
        };
        for (int i = cluster; i < p.items && !timed_out; i += clusters) {
            const OrthoTile t = ortho_tile<S, TALL>(p, i);
            timed_out = !(t.phase == kOrthoGram     ? tile(t, std::integral_constant<int, kOrthoGram>())
                          : t.phase == kOrthoSquare ? tile(t, std::integral_constant<int, kOrthoSquare>())
                                                    : tile(t, std::integral_constant<int, kOrthoUpdate>()));
        }
    }

    if (timed_out) atomicOr(p.status, kGrStatusTimeout);
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();  // nothing of the peer's is under way in this CTA's memory
    __syncwarp();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_cg<2>(tmem, S::kTmemCols);
    }
}

}  // namespace gb300
