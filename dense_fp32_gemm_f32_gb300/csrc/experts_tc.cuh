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
//   gradient of the weights: f = row k of dW, c = its column n, contraction
//               over the group's rows t: A = X, B = dY, both MN-major, read as
//               stored.  (Nothing is ragged in f and c here, and a lane that
//               holds a row's neighbouring elements packs them by itself: for
//               32 groups of 2 rows, 2048 x 4096, bound by the epilogue, 164 us
//               the other way round, 140 so, and 109 with the rest below.)
//
// float32 operands come as three bf16 parts each, x = x0 + x1 + x2 (8 bits
// each, rounded to nearest: what is left is below 2^-25 |x|), and the sum runs
// over the six products of parts that a float32 product would show; the three
// dropped ones are below 2^-24 |a||b| together.  The error grows with the number
// of additions into one accumulator (as if each cut and did not round), so
// x0 y0 has an accumulator of its own, the five small products another (256
// times smaller), and every 512 of the contraction both go to float32
// registers, which round to nearest (kGrChunk; 16-bit operands every 1024).  Measured against 64 bits, in the 2-norm,
// for a contraction of 2048: 2.1e-6 with one accumulator, 5e-7 so.
//
// Persistent CTAs (CG = 1) or CTA pairs (CG = 2: one instruction of the pair's
// first CTA multiplies 256 features by up to 256 columns, each CTA holding
// half of either operand, which halves the shared-memory fill per flop).
// Tile i goes to cluster i mod clusters.  Warps:
//   warp 0      loads: tensor-map copies of 64 k of A and B into a ring;
//   warp 1      MMAs (the pair's first CTA).  For a weight gradient the warp
//               first zeroes, in either CTA's shared memory, the rows past the
//               group's end in the slice that holds them: they are the next
//               group's, and may hold anything;
//   warp 2      schedule: which expert's rows a tile falls on, from the
//               boundary array alone (group_find: the host never needs the
//               group sizes), handed to the other warps through shared memory
//               a few tiles ahead.  The tiles of a last round that would leave
//               half of the pairs idle are split by columns among them;
//   the others  epilogue: tensor memory -> registers -> HBM, while the MMAs of
//               the next tile fill the other accumulator.
//
// Where the tiles are too few for the GPU (a token or a few, one projection), a
// cluster of 2 to 8 CTAs shares one (SPLIT): each takes a part of the
// contraction, leaves its sums in its shared memory, and adds up the columns
// that are its own from all parts, in their order.  (4 rows, 40 experts of 6690 x
// 480: 21 us on 16 SMs, 16 so.)
//
// The load and MMA warps' loops are uniform over the warp, with one elected
// lane issuing: the operands of the instructions then live in uniform
// registers.  (In a loop of one lane they do not, and moving them cost more
// than the MMAs: 775 cycles a stage of the wide tile, whose MMAs take 512.)
//
// Measured on GB300 (bf16 and even groups unless said; warm): 16 experts of 4096 x
// 4096, 16384 rows 293 us, 1.88 PFLOP/s, the rate of the library's plain product;
// the weights' gradient of the same 297 us; 32 experts of 2048 x 4096, 64 rows
// 77 us, 7.0 TB/s (the weights' bytes); 8 experts of 4096 x 2048, 8192 rows 79 us
// (dX) and 80 us (dW), 1.74 PFLOP/s, bound by the last round of tiles (83 us
// before its tiles were split; 90 with uneven groups); float32, 4 experts of 1024
// x 2048, 2048 rows 54 us with its operands' copies (15 us), 160 TFLOP/s of
// float32, six times that of bf16: two rounds of 128 tiles on 76 pairs bound it.
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
constexpr unsigned int kGrStatusTimeout = 4u;  // the library's timeout bit

// Contraction after which the accumulators go to float32 registers.  Measured:
// an instruction cuts each of its 16 products 25 bits below the largest of
// them and the accumulator, and their sum to 24 bits, so that it loses up to
// 16 * 2^-25 + 2^-23 = 6e-7 of the sum of magnitudes so far; 64 instructions
// stay below 3.9e-5 of it whatever the operands.  With one accumulator for the
// whole contraction, positive bf16 operands were off by 7.9e-5 for 16384 rows
// and 8e-4 for 131072.
template <int PARTS>
constexpr int kGrChunk = PARTS > 1 ? 512 : 1024;

struct GroupedTcParams {
    const int* offsets;
    int T, E;
    int F, C, K;        // features (weight gradient: rows of dW); its columns; forward: contraction length
    int ftiles, ctiles; // feature tiles; weight gradient: column tiles
    int a_planes;       // third coordinate of A's part p, expert e: p * a_planes + (weight gradient ? 0 : e)
    void* out;
    long long ldo, so;  // elements between rows; weight gradient: between experts
    int out_type;
    int ks;             // SPLIT: CTAs of a cluster
    int align;          // bytes that the output's rows are aligned to (2 .. 16)
    uint32_t idesc;     // instruction descriptor without the column count
    unsigned long long timeout_ns;
    unsigned int* status;
};

constexpr int kGrPatchBytes = 32 * 64;  // an epilogue warp's patch: 32 rows of 64 bytes

constexpr int kSchedSlots = 4;  // tiles that the schedule warp is ahead
constexpr int kSchedBytes = 32 * kSchedSlots, kSchedBars = 2 * kSchedSlots;

// Ring stages that fit beside `other` bytes and the barriers; 10 cover the
// latency of the narrow tiles' stages too.
constexpr int kRing(int stage, int other) {
    const int n = (227 * 1024 - 1024 - 512 - other) / stage;
    return n < 10 ? n : 10;
}

template <int TN_, int CG_, int PARTS_>
struct GroupedShape {
    static constexpr int TN = TN_, CG = CG_, PARTS = PARTS_;
    static constexpr int kCols = TN / CG;            // columns this CTA loads
    static constexpr int kABytes = 128 * 128;        // a part: 128 features x 64 k
    static constexpr int kBBytes = kCols * 128;      // a part: the columns x 64 k
    static constexpr int kStageBytes = PARTS * (kABytes + kBBytes);
    // Epilogue warps: two a quarter of the lanes for wide tiles, which short
    // contractions (weight gradients of few rows) leave to the epilogue's speed.
    static constexpr int kEpiWarps = PARTS == 1 && TN > 64 ? 8 : 4;
    static constexpr int kThreads = 32 * (3 + kEpiWarps);
    static constexpr int kPatches = kEpiWarps * kGrPatchBytes;
    static constexpr int kStages = kRing(PARTS * (kABytes + kBBytes), kPatches);
    static constexpr int kBoxCols = kCols < 64 ? kCols : 64;  // columns of a tensor-map box of B
    static constexpr int kAccCols = PARTS > 1 ? 2 * TN : TN;  // tensor-memory columns of one accumulator (pair)
    static constexpr int kTmemCols = 2 * kAccCols;
    static constexpr int kBars = 3 * kStages + 4 + kSchedBars;  // full, empty, peer_full; acc_full, acc_empty x 2
    static constexpr int kSmem = kStages * kStageBytes + kPatches + kSchedBytes + 8 * kBars + 16 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(kStages >= 2 && kBBytes % 1024 == 0, "ring");
    static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory columns");
};

struct GroupedTile {
    int valid, e, f0, c0, cols;  // c0: row t, or column of X (weight gradient)
    int k0, klen;                // weight gradient: the contraction's first row and length
    int srow;                    // MXFP4: the first column's place among the scale blocks' rows
};

// Tiles of the whole product.
template <bool WGRAD, int TN>
__device__ __forceinline__ int grouped_tiles(const GroupedTcParams& p) {
    if constexpr (WGRAD)
        return p.E * p.ftiles * p.ctiles;
    else
        return group_total(p.offsets, p.E, p.T, [&](int n) { return (n + TN - 1) / TN * p.ftiles; });
}

// Place of a group's tile `local` of `n` (row tiles) x `ftiles`: feature tiles
// in bands of 16, in which the features run fastest.  The tiles in flight then
// share a band of the weights (4096 features at most) and a few of the rows, and
// the shorter last tiles of a group fall on different clusters.  Against rows
// running fastest over the whole group: 8192^3 580 -> 546 us, 16384 x 4096 x 4096
// as one group 327 -> 312 us, over 16 uneven groups 312 -> 305 us; bands of 8
// are no faster, and bands of 4 slow even groups down (284 -> 311 us).
__device__ __forceinline__ void tile_place(int local, int n, int ftiles, int& f, int& row) {
    constexpr int kBand = 16;
    const int band = local / (kBand * n);
    const int rest = local - band * kBand * n, width = min(kBand, ftiles - band * kBand);
    row = rest / width;
    f = band * kBand + rest - row * width;
}

// Tile number `i` (there is one), from the same cursor in increasing order
// (whole warp).
template <bool WGRAD, int TN, int FT>
__device__ __forceinline__ void grouped_tile(const GroupedTcParams& p, int i, GroupCursor& cur, GroupedTile& t) {
    GroupHit h = {};
    if constexpr (WGRAD) {
        const int per = p.ftiles * p.ctiles;
        (void)group_find(p.offsets, p.E, p.T, i, cur, [&](int) { return per; }, h);
        t.f0 = h.local / p.ctiles * FT;
        t.c0 = h.local % p.ctiles * TN;
        t.cols = min(TN, p.C - t.c0);
        t.k0 = h.start;
        t.klen = h.end - h.start;
    } else {
        (void)group_find(p.offsets, p.E, p.T, i, cur, [&](int n) { return (n + TN - 1) / TN * p.ftiles; }, h);
        const int n = max(1, (h.end - h.start + TN - 1) / TN);
        int f, row;
        tile_place(h.local, n, p.ftiles, f, row);
        t.f0 = f * FT;
        t.c0 = h.start + row * TN;
        t.cols = min(TN, h.end - t.c0);
        t.k0 = 0;
        t.klen = p.K;
    }
    t.e = h.e;
    t.srow = 0;
}

// Tiles of the last, partial round over the clusters, split by columns when
// that round has at most half as many as there are clusters: item i of a
// cluster's sequence is tile i while i < full, then part (i - full) % parts of
// tile full + (i - full) / parts.
struct LastRound {
    int total, full, parts;
    // PARTS: the most parts, a divisor of the tile's columns into multiples of 64.
    template <int PARTS>
    __device__ __forceinline__ void set(int tiles, int clusters) {
        total = tiles;
        full = tiles / clusters * clusters;
        const int fit = total > full ? clusters / (total - full) : 1;
        parts = fit >= PARTS ? PARTS : PARTS == 4 && fit >= 2 ? 2 : 1;
    }
};

// The schedule warp: items first, first + step, ... into the slots at `slots`
// (barriers: a full and an empty one a slot), then one that is not valid.
// find(tile, t) fills in a tile; TN: its columns.  Whole warp; false on a
// timeout.
template <int TN, typename Find>
__device__ __forceinline__ bool sched_run(uint32_t slots, uint32_t bars, int first, int step, const LastRound& last,
                                          uint64_t tmo, Find find) {
    int n = 0;
    for (int i = first;; i += step) {
        GroupedTile t = {};
        int tile = i, part = 0;
        if (i >= last.full && last.parts > 1) {
            tile = last.full + (i - last.full) / last.parts;
            part = (i - last.full) % last.parts;
        }
        if (tile < last.total) {
            find(tile, t);
            t.valid = 1;
            if (last.parts > 1 && i >= last.full) {
                const int width = TN / last.parts, off = part * width;
                t.cols = min(width, t.cols - off);
                t.c0 += off;
                t.srow += off;
                if (t.cols <= 0) continue;
            }
        }
        const int slot = n % kSchedSlots, round = n / kSchedSlots;
        ++n;
        if (round > 0 && !mbar_wait_warp<false>(bars + 8 * (kSchedSlots + slot), (round - 1) & 1, tmo)) return false;
        if (elect_one()) {
            sts128i(slots + 32 * slot, make_int4(t.valid, t.e, t.f0, t.c0));
            sts128i(slots + 32 * slot + 16, make_int4(t.cols, t.k0, t.klen, t.srow));
            mbar_arrive(bars + 8 * slot);
        }
        __syncwarp();
        if (!t.valid) return true;
    }
}

// A consumer warp's next tile; false at the end, or (timed_out set) on a timeout.
struct SchedReader {
    uint32_t slots, bars;
    int n = 0;
    __device__ __forceinline__ bool next(GroupedTile& t, uint64_t tmo, bool& timed_out) {
        const int slot = n % kSchedSlots, round = n / kSchedSlots;
        if (!mbar_wait_warp<false>(bars + 8 * slot, round & 1, tmo)) {
            timed_out = true;
            return false;
        }
        const int4 a = lds128i(slots + 32 * slot), b = lds128i(slots + 32 * slot + 16);
        t.valid = warp_uniform(a.x), t.e = warp_uniform(a.y), t.f0 = warp_uniform(a.z), t.c0 = warp_uniform(a.w);
        t.cols = warp_uniform(b.x), t.k0 = warp_uniform(b.y), t.klen = warp_uniform(b.z), t.srow = warp_uniform(b.w);
        if (elect_one()) mbar_arrive(bars + 8 * (kSchedSlots + slot));
        __syncwarp();
        ++n;
        return t.valid != 0;
    }
};

// A weight gradient's slice with `left` rows from its first to the group's end
// whose last instruction takes rows past that end.
__device__ __forceinline__ bool grouped_tail(int left) { return left < kGrBK && (left & 15) != 0; }

// Byte `byte` of row `row` of a warp's patch.  The 16-byte pieces of a row trade
// places by the row's number, so that 8 lanes a row apart and 8 lanes two rows
// of 4 fall on all banks alike.
__device__ __forceinline__ uint32_t patch_at(uint32_t patch, int row, int byte) {
    return patch + static_cast<uint32_t>(row * 64 + ((((byte >> 4) ^ (row >> 1)) & 3) << 4) + (byte & 15));
}

// The patch's rows to the output's, G bytes a lane: rows 0 .. rows - 1 of `ld`
// elements, columns below `cols`.
template <int G, typename T>
__device__ __forceinline__ void patch_store(uint32_t patch, T* o, long long ld, int rows, int cols) {
    const int lane = threadIdx.x & 31;
    constexpr int kLanes = 64 / G, kRows = 32 / kLanes;  // lanes a row, rows an instruction
    const int byte = lane % kLanes * G, col = byte / static_cast<int>(sizeof(T));
    if (col < cols) {
        T* d = o + (lane / kLanes) * ld + col;
#pragma unroll
        for (int j = 0; j < 32; j += kRows) {
            const int r = j + lane / kLanes;
            const uint32_t from = patch_at(patch, r, byte);
            if (r < rows) {
                if constexpr (G == 16) {
                    *reinterpret_cast<float4*>(d) = lds128(from);
                } else if constexpr (G == 8) {
                    uint2 w;
                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "r"(from) : "memory");
                    *reinterpret_cast<uint2*>(d) = w;
                } else if constexpr (G == 4) {
                    uint32_t w;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(from) : "memory");
                    *reinterpret_cast<uint32_t*>(d) = w;
                } else {
                    unsigned short w;
                    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(w) : "r"(from) : "memory");
                    *reinterpret_cast<unsigned short*>(d) = w;
                }
            }
            d += kRows * ld;
        }
    }
}

// The widest stores that the rows' alignment (`align` bytes, 2 .. 16) and the
// number of columns allow.
template <typename T>
__device__ __forceinline__ void patch_store_any(uint32_t patch, int align, T* o, long long ld, int rows, int cols) {
    constexpr int kAll = 64 / sizeof(T);
    const int odd = (cols >= kAll ? 0 : cols) * static_cast<int>(sizeof(T));  // bytes of a row's last columns
    if (align == 16 && odd % 16 == 0)
        patch_store<16>(patch, o, ld, rows, cols);
    else if (align >= 8 && odd % 8 == 0)
        patch_store<8>(patch, o, ld, rows, cols);
    else if (sizeof(T) == 4 || (align >= 4 && odd % 4 == 0))
        patch_store<4>(patch, o, ld, rows, cols);
    else
        patch_store<2>(patch, o, ld, rows, cols);
}

template <typename V>
__device__ __forceinline__ float as_f32(V v) {
    if constexpr (__is_same(V, float))
        return v;
    else
        return __uint_as_float(v);
}

// A warp's 32 features x 32 columns, a feature a lane, to the output's rows,
// of which each column is one (columns 0 .. n - 1; features below `features`).
// float32 goes out directly, 128 bytes an instruction; 2-byte elements would
// be 64, so they pass through the patch.
template <typename T, typename V>
__device__ __forceinline__ void store_features(uint32_t patch, int align, T* o, long long ld, const V* v, int n,
                                               int features) {
    const int lane = threadIdx.x & 31;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const T x = from_f32<T>(as_f32(v[j]));
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(patch_at(patch, j, lane * 2)),
                         "h"(*reinterpret_cast<const unsigned short*>(&x))
                         : "memory");
        }
        __syncwarp();
        patch_store_any(patch, align, o, ld, n, features);
        __syncwarp();
    } else {
        T* d = o + lane;
        if (lane >= features) n = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j < n) *d = as_f32(v[j]);
            d += ld;
        }
    }
}

// A warp's 32 rows x 32 columns, a row a lane, to the output (rows 0 .. rows -
// 1, columns below `cols`): through the patch, 64 bytes of each row at a time.
template <typename T, typename V>
__device__ __forceinline__ void store_rows(uint32_t patch, int align, T* o, long long ld, const V* v, int rows,
                                           int cols) {
    const int lane = threadIdx.x & 31;
    constexpr int kStep = 64 / sizeof(T);
#pragma unroll
    for (int c = 0; c < 32; c += kStep) {
        if (c < cols) {  // (warp-uniform)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (sizeof(T) == 4) {
                        w[j] = __float_as_uint(as_f32(v[c + 4 * i + j]));
                    } else {
                        w[j] = pair_from_f32<T>(as_f32(v[8 * i + 2 * j]), as_f32(v[8 * i + 2 * j + 1]));
                    }
                }
                sts128i(patch_at(patch, lane, 16 * i), make_int4(w[0], w[1], w[2], w[3]));
            }
            __syncwarp();
            patch_store_any(patch, align, o + c, ld, rows, cols - c);
            __syncwarp();
        }
    }
}

// `at`: the element of the first row and column.  ONLY_F32: the output is
// (float32 operands).  ROWS: a lane holds a row of
// the output (else a feature); n rows, `cols` columns are there.
template <bool ROWS, bool ONLY_F32 = false, typename P, typename V>
__device__ __forceinline__ void grouped_store(const P& p, uint32_t patch, long long at, const V* v, int n, int cols) {
    auto typed = [&](auto zero) {
        using T = decltype(zero);
        T* const o = static_cast<T*>(p.out) + at;
        if constexpr (ROWS)
            store_rows(patch, p.align, o, p.ldo, v, n, cols);
        else
            store_features(patch, p.align, o, p.ldo, v, n, cols);
    };
    if (ONLY_F32 || p.out_type == 0)
        typed(0.f);
    else if constexpr (!ONLY_F32) {
        if (p.out_type == 1)
            typed(__nv_bfloat16());
        else
            typed(__half());
    }
}

// The split form: this CTA's part of a tile's contraction, in whole stages.
__device__ __forceinline__ void split_contraction(GroupedTile& t, int part, int parts, int stage) {
    const int per = ((t.klen + stage - 1) / stage + parts - 1) / parts * stage;
    const int from = min(t.klen, part * per);
    t.k0 = from;
    t.klen = min(t.klen, from + per) - from;
}

// Its sums, columns c .. c + 31 of feature f, to the (idle) ring: a column a
// row of 128.
template <typename V>
__device__ __forceinline__ void leave_part(uint32_t ring, int c, int f, const V (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(ring + static_cast<uint32_t>(((c + j) * 128 + f) * 4)),
                     "f"(as_f32(v[j]))
                     : "memory");
}

// The columns that are this CTA's, part p of `parts` every `parts`-th, from
// all CTAs of the cluster.
template <typename P>
__device__ __forceinline__ void add_parts(const P& p, uint32_t ring, const GroupedTile& t, int part, int parts,
                                          int thread, int threads) {
    const int f = thread & 127;
    if (t.f0 + f >= p.F) return;
    for (int c = part + parts * (thread >> 7); c < t.cols; c += parts * (threads >> 7)) {
        const uint32_t at = ring + static_cast<uint32_t>((c * 128 + f) * 4);
        float s = 0.f;
        for (int q = 0; q < parts; ++q) s += ld_shared_cluster_f32(map_shared_rank(at, q));
        const long long o = (t.c0 + c) * p.ldo + t.f0 + f;
        if (p.out_type == 0)
            static_cast<float*>(p.out)[o] = s;
        else if (p.out_type == 1)
            static_cast<__nv_bfloat16*>(p.out)[o] = from_f32<__nv_bfloat16>(s);
        else
            static_cast<__half*>(p.out)[o] = from_f32<__half>(s);
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

// AMN, BMN: the operand is MN-major in HBM and shared memory (else K-major);
// both: a weight gradient.
template <bool AMN, bool BMN, int TN, int CG, int PARTS, bool SPLIT = false>
__global__ void __launch_bounds__(GroupedShape<TN, CG, PARTS>::kThreads, 1)
    grouped_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const GroupedTcParams p) {
    using S = GroupedShape<TN, CG, PARTS>;
    constexpr bool WGRAD = AMN && BMN;
    static_assert(!BMN || (AMN && S::kCols % 64 == 0), "the weight gradient's columns come in blocks of 64");
    static_assert(!SPLIT || (CG == 1 && PARTS == 1 && !BMN && S::kStages * S::kStageBytes >= TN * 128 * 4), "split form");
    constexpr int FT = 128 * CG;
    constexpr bool PAIR = CG == 2;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t baseB = base + PARTS * S::kABytes;  // B's parts follow A's in a stage
    const uint32_t patches = base + S::kStages * S::kStageBytes;
    const uint32_t slots = patches + S::kPatches;
    const uint32_t bars = slots + kSchedBytes;
    const uint32_t full0 = bars, empty0 = bars + 8 * S::kStages, peer0 = bars + 16 * S::kStages;
    const uint32_t acc_full0 = bars + 24 * S::kStages, acc_empty0 = acc_full0 + 16, sched0 = acc_empty0 + 16;
    const uint32_t tmem_slot = bars + 8u * S::kBars;

    const int warp = warp_uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int rank = PAIR ? warp_uniform(static_cast<int>(cluster_ctarank())) : 0;
    const int share = SPLIT ? p.ks : CG;  // CTAs of a tile
    const int part = SPLIT ? warp_uniform(static_cast<int>(cluster_ctarank())) : 0;
    const int cluster = static_cast<int>(blockIdx.x) / share, clusters = static_cast<int>(gridDim.x) / share;
    const unsigned long long tmo = p.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
            mbar_init(peer0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full0 + 8 * b, 1);
            mbar_init(acc_empty0 + 8 * b, S::kEpiWarps * CG);
        }
        for (int j = 0; j < kSchedSlots; ++j) {
            mbar_init(sched0 + 8 * j, 1);
            mbar_init(sched0 + 8 * (kSchedSlots + j), 2 + S::kEpiWarps);  // load, MMA and epilogue warps
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
    grid_dependency_wait();  // the set-up above ran beside the end of the kernel before

    bool timed_out = false;
    GroupedTile t, split = {};  // split: the tile whose parts this cluster has to add up
    SchedReader tiles{slots, sched0};
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        const uint32_t bar0 = PAIR ? warp_uniform(map_shared_rank(full0, 0)) : full0;
        const bool issuer = elect_one();
        uint32_t s = 0, phase = 1;  // (the first round finds every stage empty)
        int issued = 0;
        while (!timed_out && tiles.next(t, tmo, timed_out)) {
            const int cols = (t.cols + 15) & ~15;    // columns of the instruction,
            const int mine = cols / CG;              // this CTA's part of them
            const int c0 = t.c0 + rank * mine, f0 = t.f0 + rank * 128;
            const int boxes = (mine + S::kBoxCols - 1) / S::kBoxCols;
            constexpr uint32_t kBox = S::kBoxCols * 128;
            const uint32_t bytes = PARTS * (S::kABytes + boxes * kBox);
            const int pa = WGRAD ? 0 : t.e;
            for (int k = 0; k < t.klen; k += kGrBK) {
                if (!mbar_wait_warp<false>(empty0 + 8 * s, phase, tmo)) {
                    timed_out = true;
                    break;
                }
                // A pair's loads all arrive on the first CTA's barrier, but
                // for a slice with rows past the group's end that the second
                // CTA has to zero first.
                const bool own = !PAIR || (WGRAD && grouped_tail(t.klen - k));
                const uint32_t bar = (own ? full0 : bar0) + 8 * s;
                const uint32_t a = base + s * S::kStageBytes, b = baseB + s * S::kStageBytes;
                const int kc = t.k0 + k;
                if (issuer) {
                    if (own)
                        mbar_arrive_expect_tx(full0 + 8 * s, bytes);
                    else if (rank == 0)
                        mbar_arrive_expect_tx(full0 + 8 * s, 2 * bytes);
                    auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, int z) {
                        if constexpr (PAIR)
                            tma_load_3d_pair(dst, map, bar, x, y, z);
                        else
                            tma_load_3d(dst, map, bar, x, y, z);
                    };
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        if constexpr (AMN) {
                            load(a + part * S::kABytes, &tmA, f0, kc, part * p.a_planes + pa);
                            load(a + part * S::kABytes + 64 * 128, &tmA, f0 + 64, kc, part * p.a_planes + pa);
                        } else {
                            load(a + part * S::kABytes, &tmA, kc, f0, part * p.a_planes + pa);
                        }
#pragma unroll
                        for (int j = 0; j < S::kCols / S::kBoxCols; ++j) {
                            if (j < boxes) {
                                if constexpr (BMN)
                                    load(b + part * S::kBBytes + j * kBox, &tmB, c0 + S::kBoxCols * j, kc, part);
                                else
                                    load(b + part * S::kBBytes + j * kBox, &tmB, kc, c0 + S::kBoxCols * j, part);
                            }
                        }
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
        const uint64_t descA = AMN ? umma_desc_mnmajor_sw128(base, 64 * 128) : umma_desc_kmajor_sw128(base);
        const uint64_t descB = BMN ? umma_desc_mnmajor_sw128(baseB, 64 * 128) : umma_desc_kmajor_sw128(baseB);
        // 16 k: 32 bytes of each row (K-major), 16 rows of 128 bytes (MN-major); addresses in units of 16
        constexpr uint32_t ka = AMN ? 128 : 2, kb = BMN ? 128 : 2;
        constexpr uint32_t pa = S::kABytes / 16, pb = S::kBBytes / 16;
        const uint32_t peer_empty0 = PAIR ? warp_uniform(map_shared_rank(empty0, 1)) : 0;
        const uint32_t peer_acc_full0 = PAIR ? warp_uniform(map_shared_rank(acc_full0, 1)) : 0;
        const uint32_t lead_peer0 = PAIR ? warp_uniform(map_shared_rank(peer0, 0)) : 0;
        const bool issuer = elect_one();
        uint32_t s = 0, phase = 0;
        uint32_t tails = 0;  // bit s: parity of the slices with rows to zero so far in stage s
        int unit = 0;        // accumulators filled
        auto next = [&] {
            if (++s == S::kStages) {
                s = 0;
                phase ^= 1;
            }
        };
        while (!timed_out && tiles.next(t, tmo, timed_out)) {
            if (rank != 0 && !WGRAD) continue;  // (the first CTA issues for both)
            const uint32_t idesc = p.idesc | static_cast<uint32_t>((t.cols + 15) >> 4) << 18;
            const bool tail = WGRAD && grouped_tail(t.klen % kGrBK ? t.klen % kGrBK : kGrBK);
            constexpr int chunk = kGrChunk<PARTS>;
            int k = 0;
            do {
                const int buf = unit & 1;
                const uint32_t acc = tmem + static_cast<uint32_t>(buf * S::kAccCols);
                const int end = min(t.klen, k + chunk);
                const int plain = tail && end == t.klen ? end / kGrBK * kGrBK : end;  // slices up to here: as they are
                bool more = false;  // the accumulators hold something
                auto slice = [&](int left) {
                    const uint32_t off = s * (S::kStageBytes / 16);
                    const uint64_t a = descA + off, b = descB + off;
                    if (issuer) {
#pragma unroll
                        for (int kk = 0; kk < kGrBK / 16; ++kk) {
                            if (left > kk * 16) {
                                const bool add = more || kk > 0;
                                if constexpr (PARTS == 1) {
                                    umma_f16<CG>(acc, a + kk * ka, b + kk * kb, idesc, add);
                                } else {
                                    auto mma = [&](uint32_t d, int i, int j, bool sum) {
                                        umma_f16<CG>(d, a + i * pa + kk * ka, b + j * pb + kk * kb, idesc, sum);
                                    };
                                    mma(acc + TN, 2, 0, add);
                                    mma(acc + TN, 1, 1, true);
                                    mma(acc + TN, 0, 2, true);
                                    mma(acc + TN, 1, 0, true);
                                    mma(acc + TN, 0, 1, true);
                                    mma(acc, 0, 0, add);
                                }
                            }
                        }
                        umma_commit_cg<CG>(empty0 + 8 * s);
                        if constexpr (PAIR) umma_commit_cg<CG>(peer_empty0 + 8 * s);
                    }
                    __syncwarp();
                    more = true;
                };
                if (rank == 0) {
                    if (unit >= 2 && !mbar_wait_warp<PAIR>(acc_empty0 + 8 * buf, ((unit >> 1) - 1) & 1, tmo))
                        timed_out = true;
                    tc_fence_after_sync();
                    for (int q = k; q < plain && !timed_out; q += kGrBK) {
                        if (!mbar_wait_warp<false>(full0 + 8 * s, phase, tmo)) {
                            timed_out = true;
                            break;
                        }
                        tc_fence_after_sync();
                        slice(end - q);
                        next();
                    }
                } else {
                    for (int q = k; q < plain; q += kGrBK) next();
                }
                if constexpr (WGRAD) {
                    if (plain < end && !timed_out) {
                        // The last slice: rows left .. of its last instruction's
                        // 16 belong to others.  Zeros (rows of 128 bytes in
                        // blocks of 64 rows, A's and B's).
                        const int left = end - plain, past = (left + 15) & ~15;
                        const uint32_t full_phase = rank != 0 ? tails >> s & 1 : phase;
                        if (!mbar_wait_warp<false>(full0 + 8 * s, full_phase, tmo)) timed_out = true;
                        constexpr int blocks = S::kStageBytes / (64 * 128);
                        for (int row = left + (lane >> 3); row < past; row += 4)
#pragma unroll
                            for (int b = 0; b < blocks; ++b)
                                sts128(base + s * S::kStageBytes + static_cast<uint32_t>(b * 64 * 128 + row * 128 + (lane & 7) * 16),
                                       make_float4(0.f, 0.f, 0.f, 0.f));
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (!timed_out) {
                            if (rank != 0) {
                                if (issuer) mbar_arrive_cluster(lead_peer0 + 8 * s);
                                __syncwarp();
                            } else {
                                if (PAIR && !mbar_wait_warp<true>(peer0 + 8 * s, tails >> s & 1, tmo)) timed_out = true;
                                tc_fence_after_sync();
                                if (!timed_out) slice(left);
                            }
                        }
                        tails ^= 1u << s;
                        next();
                    }
                }
                if (timed_out) break;
                if (rank == 0 && issuer) {
                    umma_commit_cg<CG>(acc_full0 + 8 * buf);
                    if constexpr (PAIR) umma_commit_cg<CG>(peer_acc_full0 + 8 * buf);
                }
                __syncwarp();
                ++unit;
                k = end;
            } while (k < t.klen);
        }
        if (timed_out && rank == 0) {  // the MMAs in flight end before tensor memory is freed
            if (issuer) umma_commit_cg<CG>(acc_full0 + 8 * (unit & 1));
            __syncwarp();
            (void)mbar_wait_warp<false>(acc_full0 + 8 * (unit & 1), (unit >> 1) & 1, tmo);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ schedule
        GroupCursor cur = group_begin(p.offsets, p.T);
        LastRound last;
        last.set<(PAIR ? TN / 64 : 1)>(grouped_tiles<WGRAD, TN>(p), clusters);
        if (!sched_run<TN>(slots, sched0, cluster, clusters, last, tmo,
                           [&](int i, GroupedTile& u) {
                               grouped_tile<WGRAD, TN, FT>(p, i, cur, u);
                               if constexpr (SPLIT) split_contraction(u, part, p.ks, kGrBK);
                           }))
            timed_out = true;
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;
        const uint32_t acc_empty_lead = PAIR ? warp_uniform(map_shared_rank(acc_empty0, 0)) : acc_empty0;
        const int half = (warp - 3) >> 2;  // of the chunks of 32 columns, every second one each
        if (!WGRAD) {
            const int worker = static_cast<int>(blockIdx.x) * S::kEpiWarps + warp - 3;
            const int workers = static_cast<int>(gridDim.x) * S::kEpiWarps;
            if (p.out_type == 0)
                grouped_zero_rows<float>(p, worker, workers);
            else  // (bf16 and f16 zeros are the same bits)
                grouped_zero_rows<__half>(p, worker, workers);
        }
        int unit = 0;
        while (!timed_out && tiles.next(t, tmo, timed_out)) {
            const int f = t.f0 + rank * 128 + 32 * q;  // the warp's first feature (weight gradient: row)
            const uint32_t patch = patches + (warp - 3) * kGrPatchBytes;
            auto store = [&](int c, const auto* v) {
                if constexpr (WGRAD)
                    grouped_store<true, (PARTS > 1)>(p, patch, t.e * p.so + f * p.ldo + t.c0 + c, v, p.F - f, t.cols - c);
                else
                    grouped_store<false, (PARTS > 1)>(p, patch, (t.c0 + c) * p.ldo + f, v, t.cols - c, p.F - f);
            };
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
            constexpr int kStep = 8 * S::kEpiWarps;  // the warp's columns: 32 of every kStep, from 32 `half` on
            uint32_t acc;
            if constexpr (PARTS == 1) {
                if (!wait(acc)) {
                    timed_out = true;
                    break;
                }
                if (t.klen > kGrChunk<PARTS>) {
                    // All accumulators' sums, left in the last.  (So the stores below have the
                    // registers to themselves; 16 columns a load for the same reason.  8 experts of
                    // 2048 x 2048 by 8192 rows: 288 us with one accumulator, 291 so.)
                    float sum[TN / kStep][32] = {};
                    for (int k = kGrChunk<PARTS>;; k += kGrChunk<PARTS>) {
#pragma unroll
                        for (int i = 0; i < TN / kStep; ++i) {
                            const int c = 32 * half + kStep * i;
                            if (c < t.cols) {
#pragma unroll
                                for (int h = 0; h < 32; h += 16) {
                                    uint32_t v[16];
                                    __syncwarp();
                                    tmem_ld_32x32b_x16(acc + static_cast<uint32_t>(c + h), v);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int j = 0; j < 16; ++j) sum[i][h + j] += __uint_as_float(v[j]);
                                }
                            }
                        }
                        if (k >= t.klen) break;
                        release();
                        if (!wait(acc)) {
                            timed_out = true;
                            break;
                        }
                    }
                    if (timed_out) break;
#pragma unroll
                    for (int i = 0; i < TN / kStep; ++i) {
                        const int c = 32 * half + kStep * i;
                        if (c < t.cols) {
#pragma unroll
                            for (int h = 0; h < 32; h += 16) {
                                uint32_t v[16];
#pragma unroll
                                for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(sum[i][h + j]);
                                __syncwarp();
                                tmem_st_32x32b_x16(acc + static_cast<uint32_t>(c + h), v);
                            }
                        }
                    }
                    tmem_wait_st();
                }
                for (int c = 32 * half; c < t.cols; c += kStep) {
                    uint32_t v[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(c), v);
                    tmem_wait_ld();
                    if ((WGRAD || SPLIT) && t.klen == 0) {  // no MMA wrote the accumulator
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0;
                    }
                    if constexpr (SPLIT)
                        leave_part(base, c, 32 * q + lane, v);
                    else
                        store(c, v);
                }
                if constexpr (SPLIT) split = t;
                release();
            } else {
                float sum[TN];
#pragma unroll
                for (int j = 0; j < TN; ++j) sum[j] = 0.f;
                for (int k = 0; k < t.klen || k == 0; k += kGrChunk<PARTS>) {
                    if (!wait(acc)) {
                        timed_out = true;
                        break;
                    }
                    if (t.klen > 0) {
#pragma unroll
                        for (int c = 0; c < TN; c += 32) {
                            if (c < t.cols) {
                                uint32_t v[32], w[32];
                                tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(TN + c), w);
                                tmem_ld_32x32b_x32(acc + static_cast<uint32_t>(c), v);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    sum[c + j] += __uint_as_float(v[j]) + __uint_as_float(w[j]);
                            }
                        }
                    }
                    release();
                }
                if (timed_out) break;
#pragma unroll
                for (int c = 0; c < TN; c += 32)
                    if (c < t.cols) store(c, sum + c);
                __syncwarp();
            }
        }
    }

    if (timed_out) atomicOr(p.status, kGrStatusTimeout);
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();  // nothing of the peer's is under way in this CTA's memory
    if constexpr (SPLIT) {
        cluster_sync_all();  // every part is there
        if (warp >= 3 && split.valid && !timed_out)
            add_parts(p, base, split, part, p.ks, (warp - 3) * 32 + lane, 32 * S::kEpiWarps);
        cluster_sync_all();  // and has been read
    }
    __syncwarp();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_cg<CG>(tmem, S::kTmemCols);
    }
}

}  // namespace gb300
