// MXFP4 quantisation and its inverse.
//
// A block of 32 columns shares the scale 2^s, s = floor(log2 m) - 2 for its
// largest magnitude m: m 2^-s lies in [4, 8), next to the largest 4-bit value
// 6 = 1.5 * 2^2.  The exponent field of m's bits gives s without a logarithm,
// and m is taken over the bits as integers, in which a NaN counts as larger
// than any number.
//
// Both kernels move bytes and compute next to nothing.  A warp takes one row
// and up to 1024 of its columns, 8 columns a lane and step: 16-byte loads (two
// for float32), the block's maximum by two shuffles among 4 lanes, 4 bytes of
// codes a lane (128 contiguous bytes a warp) and the 4 scales of 128 columns
// as one 4-byte word.  All of a warp's loads are issued before the first use.
// Measured: quantise 16384 x 4096 bf16 30 us (5.7 TB/s; the instructions still
// show beside the bytes' 25 us), 8192 x 8192 float32 45 us
// (6.8 TB/s, the copy's rate); read back 27 us (6.2 TB/s) and 47 us (6.5 TB/s).
// A warp for 512 columns instead: 36 us, for 2048: 78 us before the loads were
// made one batch.
#include "../../include/sgemm_experts.h"
#include "experts.h"
#include "experts_groups.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kSteps = 4;               // steps of 256 columns a warp takes
constexpr int kCols = 256 * kSteps;     // columns a warp takes
constexpr int kWarps = 4;               // warps a CTA

// Eight float32 to eight codes, the first in the low bits: to nearest, ties to
// the even code, magnitudes beyond 6 to 6.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight codes to eight float32 (exact).
__device__ __forceinline__ void from_e2m1x8(uint32_t c, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 x = *reinterpret_cast<const __half2*>(&h[i]);
        v[2 * i] = __low2float(x);
        v[2 * i + 1] = __high2float(x);
    }
}

// Columns c .. c + 7 of a row of K, as they lie; zeros past the row's end.
// WHOLE: all 8 are there, on the 16-byte grid.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
};

template <bool WHOLE, typename T>
__device__ __forceinline__ void load8(const T* row, int c, int K, bool vec, Raw8<T>& r) {
    constexpr int n = 16 / sizeof(T);
    if (WHOLE || (vec && c + 8 <= K)) {
#pragma unroll
        for (int h = 0; h < 8 / n; ++h) r.w[h] = __ldg(reinterpret_cast<const uint4*>(row + c) + h);
    } else {
        T* t = reinterpret_cast<T*>(&r);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = c + i < K ? row[c + i] : from_f32<T>(0.f);
    }
}

// The exponent field (as of float32) of the largest magnitude among a block's
// 32 values, 8 in each of 4 neighbouring lanes; 255 with an infinity or a NaN.
// Magnitudes compare as integers, 16-bit ones two at a time.
__device__ __forceinline__ uint32_t block_exponent(const Raw8<float>& r) {
    const uint32_t* t = reinterpret_cast<const uint32_t*>(&r);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, t[i] & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return m >> 23;
}

template <typename T>
__device__ __forceinline__ uint32_t block_exponent(const Raw8<T>& r) {
    static_assert(sizeof(T) == 2, "16-bit values");
    const uint32_t* t = reinterpret_cast<const uint32_t*>(&r);
    uint32_t m = t[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __vmaxu2(m, t[i] & 0x7fff7fffu);
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = max(m & 0xffffu, m >> 16);
    if constexpr (__is_same(T, __nv_bfloat16))
        return m >> 7;
    else
        return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m)))) >> 23;
}

template <typename T>
__device__ __forceinline__ void store8(T* row, int c, int K, bool vec, const float (&v)[8]) {
    if (sizeof(T) == 4 && vec && c + 8 <= K && (reinterpret_cast<uintptr_t>(row) & 31) == 0) {
        // (32 bytes a lane at once: two 16-byte stores write half sectors, 66 us instead of 47 for 8192 x 8192)
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + c), "f"(v[0]), "f"(v[1]),
                     "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                     : "memory");
    } else if (vec && c + 8 <= K) {
        constexpr int n = 16 / sizeof(T);
#pragma unroll
        for (int h = 0; h < 8 / n; ++h) {
            uint4 w;
            T* t = reinterpret_cast<T*>(&w);
#pragma unroll
            for (int i = 0; i < n; ++i) t[i] = from_f32<T>(v[h * n + i]);
            *reinterpret_cast<uint4*>(row + c + h * n) = w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < K) row[c + i] = from_f32<T>(v[i]);
    }
}

// What a warp works on: a matrix, a row, the row's place among the scale
// blocks' rows (< 0: a row of no expert) and its first column.
struct Work {
    int matrix, row, col;
    long long scale_row;
};

// A CTA takes kWarps rows (numbered over all matrices) of one chunk of
// columns.  (32-bit divisions, and one a CTA: 64-bit ones in every warp cost 3 us
// of 57 for 16384 x 4096 bf16.)
__device__ __forceinline__ bool find_work(const QuantParams& p, Work& w) {
    const unsigned chunks = (static_cast<unsigned>(p.K) + kCols - 1) / kCols;
    const unsigned block = chunks == 1 ? blockIdx.x : blockIdx.x / chunks;
    const unsigned r = block * kWarps + (threadIdx.x >> 5);
    const bool in = r < static_cast<unsigned>(p.batch) * static_cast<unsigned>(p.rows);
    w.col = static_cast<int>(blockIdx.x - block * chunks) * kCols;
    w.matrix = p.batch == 1 ? 0 : static_cast<int>(r / static_cast<unsigned>(p.rows));
    w.row = static_cast<int>(r - static_cast<unsigned>(w.matrix) * static_cast<unsigned>(p.rows));
    w.scale_row = w.row;
    if (p.offsets) {
        // The first warp's group is most often the others' too: one search a
        // CTA (36 us with one a warp for 16384 x 4096 bf16 of 8 experts, 34 so).
        __shared__ GroupHit shared;
        GroupCursor c = group_begin(p.offsets, p.rows);
        GroupHit h = {0, 0, 0, 0, 0};
        auto find = [&] {
            return w.row >= c.start &&
                   group_find(p.offsets, p.E, p.rows, w.row - c.start, c, [](int n) { return n; }, h);
        };
        if (threadIdx.x < 32) {
            const bool ok = find();
            if (threadIdx.x == 0) shared = ok ? h : GroupHit{0, 0, 0, 0, 0};
        }
        __syncthreads();
        h = shared;
        if (w.row >= h.start && w.row < h.end)
            w.scale_row = 128ll * h.block0 + (w.row - h.start);
        else
            w.scale_row = threadIdx.x >= 32 && in && find() ? 128ll * h.block0 + h.local : -1;
    }
    return in;
}

// Word of the 4 scales of columns 128 q .. of a scale row.
__device__ __forceinline__ long long scale_word(long long scale_row, int q, int kq) {
    return ((scale_row >> 7) * kq + q) * 128 + (scale_row & 31) * 4 + ((scale_row & 127) >> 5);
}

template <bool WHOLE, typename T>
__device__ __forceinline__ void quantize_row(const QuantParams& p, const Work& w, const T* row, bool vec) {
    const int lane = threadIdx.x & 31;
    const int kb = (p.K + 31) / 32, kq = (kb + 3) / 4;
    uint8_t* codes = p.codes + (static_cast<long long>(w.matrix) * p.rows + w.row) * 16 * kb;
    const long long nb = (p.rows + 127) / 128;
    uint32_t* scales = reinterpret_cast<uint32_t*>(p.scales) + w.matrix * nb * kq * 128;
    // (All loads before the first use: 54 -> 40 us for 16384 x 4096 bf16.)
    Raw8<T> raw[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) load8<WHOLE>(row, w.col + 256 * s + 8 * lane, p.K, vec, raw[s]);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int c = w.col + 256 * s + 8 * lane;
        if (!WHOLE && w.col + 256 * s >= 32 * kb) break;  // (warp-uniform)
        const uint32_t field = block_exponent(raw[s]);    // floor(log2 m) + 127
        const uint32_t byte = field == 255 ? 255 : field > 2 ? field - 2 : 0;
        // 2^-s = 2^(127 - byte).  (A block that stands for NaN: any factor, any codes.)
        const float f = __uint_as_float((254u - byte) << 23);
        const T* t = reinterpret_cast<const T*>(&raw[s]);
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = to_f32(t[i]) * f;
        if (WHOLE || c < 32 * kb) *reinterpret_cast<uint32_t*>(codes + (c >> 1)) = to_e2m1x8(u);
        uint32_t word = byte << (8 * ((lane >> 2) & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        if ((lane & 15) == 0 && (WHOLE || c < p.K) && w.scale_row >= 0)
            scales[scale_word(w.scale_row, c >> 7, kq)] = word;
    }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) quantize_kernel(const QuantParams p) {
    grid_dependency_launch();
    Work w;
    if (!find_work(p, w)) return;
    const T* row = static_cast<const T*>(p.X) + w.matrix * p.sx + w.row * p.ldx;
    const bool vec = (reinterpret_cast<uintptr_t>(row) & 15) == 0;
    if (vec && w.col + kCols <= p.K)
        quantize_row<true>(p, w, row, true);
    else
        quantize_row<false>(p, w, row, vec);
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) dequantize_kernel(const QuantParams p) {
    Work w;
    if (!find_work(p, w)) return;
    const int lane = threadIdx.x & 31;
    const int kb = (p.K + 31) / 32, kq = (kb + 3) / 4;
    T* row = static_cast<T*>(p.Y) + w.matrix * p.sy + w.row * p.ldy;
    const bool vec = (reinterpret_cast<uintptr_t>(row) & 15) == 0;
    const uint8_t* codes = p.codes_in + (static_cast<long long>(w.matrix) * p.rows + w.row) * 16 * kb;
    const long long nb = (p.rows + 127) / 128;
    const uint32_t* scales = reinterpret_cast<const uint32_t*>(p.scales_in) + w.matrix * nb * kq * 128;
    uint32_t code[kSteps], word[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int c = w.col + 256 * s + 8 * lane;
        const bool in = c < p.K && w.scale_row >= 0;
        code[s] = in ? __ldg(reinterpret_cast<const uint32_t*>(codes + (c >> 1))) : 0;
        word[s] = in ? __ldg(scales + scale_word(w.scale_row, c >> 7, kq)) : 0;
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int c = w.col + 256 * s + 8 * lane;
        if (c >= p.K) continue;
        const uint32_t byte = (word[s] >> (8 * ((lane >> 2) & 3))) & 255;
        const float f = __uint_as_float(byte == 255 ? 0x7fffffffu : byte == 0 ? 0x00400000u : byte << 23);
        float v[8];
        from_e2m1x8(code[s], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= f;
        store8(row, c, p.K, vec, v);
    }
}

template <typename K>
int launch(K kernel, const QuantParams& p, cudaStream_t s) {
    const long long rows = static_cast<long long>(p.batch) * p.rows;
    const long long ctas = (rows + kWarps - 1) / kWarps * ((p.K + kCols - 1) / kCols);
    if (ctas == 0) return SGEMM_OK;
    if (ctas > 0x7fffffffll || rows > 0xffffff00ll) return SGEMM_ERR_INVALID_ARG;
    kernel<<<static_cast<unsigned>(ctas), 32 * kWarps, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}

}  // namespace

int mxfp4_quantize(const QuantParams& p, int type, cudaStream_t s) {
    return type == SGEMM_TYPE_F32    ? launch(quantize_kernel<float>, p, s)
           : type == SGEMM_TYPE_BF16 ? launch(quantize_kernel<__nv_bfloat16>, p, s)
                                     : launch(quantize_kernel<__half>, p, s);
}

int mxfp4_dequantize(const QuantParams& p, int type, cudaStream_t s) {
    return type == SGEMM_TYPE_F32    ? launch(dequantize_kernel<float>, p, s)
           : type == SGEMM_TYPE_BF16 ? launch(dequantize_kernel<__nv_bfloat16>, p, s)
                                     : launch(dequantize_kernel<__half>, p, s);
}

}  // namespace gb300
