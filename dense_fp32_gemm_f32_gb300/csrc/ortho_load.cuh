// Elements of an update on their way to the products of ortho_tc.cuh and
// ortho_small.cu: loads, sums of squares, and X = G / (norm + eps) times 2^13 in
// two f16 parts, hi = f16(x) and lo = f16(x - hi), together 22 bits.
#pragma once

#include "experts_groups.cuh"

namespace gb300 {

// Eight neighbouring values of a row with `left` of them there.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, bool vec, float (&v)[8]) {
    if (vec && left >= 8) {
        alignas(16) T x[8];
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
            reinterpret_cast<uint4*>(x)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f32(p[i]) : 0.f;
    }
}

// Eight values each from N places, `step` octs apart from oct `first` on, of rows of `octs` octs (`cols` elements); zeros
// from oct `n` on.  whole: every oct is a vector (no oct of a row is cut short), and all loads are one without a branch
// between them (with one, 4 loads of a thread followed one another: 134 MB of bf16 54 us).
template <int N, typename T>
__device__ __forceinline__ void load_octs(const T* G, long long ld, int first, int step, int octs, int cols, int n, bool whole,
                                          bool vec, float (&v)[N][8]) {
    if (whole) {
        alignas(16) T x[N][8];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int at = min(first + u * step, n - 1), r = at / octs;
            const uint4* from = reinterpret_cast<const uint4*>(G + r * ld + (at - r * octs) * 8);
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(x[u])[i] = __ldg(from + i);
        }
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = first + u * step < n ? to_f32(x[u][i]) : 0.f;
    } else {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int at = first + u * step, r = at / octs, c = (at - r * octs) * 8;
            load8(G + r * ld + c, at < n ? cols - c : 0, vec, v[u]);
        }
    }
}

// The sum of the squares of N times eight values.  They are scaled by a power of
// two that brings the largest near 1, their squares summed in float32, and the sum
// scaled back in 64 bits: no square overflows or vanishes.  (64 bits run at 2 lanes
// a cycle of an SM: once in 32 values 8 matrices of 2048 x 4096 bf16 are read at
// the memory's speed, once in 8 the sums took 50 us.)
template <int N>
__device__ __forceinline__ double squares(const float (&v)[N][8]) {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 8 * N; ++i) most = fmaxf(most, fabsf(v[i / 8][i % 8]));  // (a NaN is passed over here and summed below)
    // 2^up brings it to [1, 2) or, from below 2^-126 or above, near that
    const int up = most > 0.f ? min(126, 127 - static_cast<int>(__float_as_uint(most) >> 23)) : 0;
    const float scale = __uint_as_float(static_cast<uint32_t>(max(up, -126) + 127) << 23);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8 * N; ++i) {
        const float x = v[i / 8][i % 8] * scale;
        s = fmaf(x, x, s);
    }
    // (s is 0 or above 2^-50, below 2^10, and 2^-2up within a double's range)
    return s * __longlong_as_double(static_cast<long long>(1023 - 2 * max(up, -126)) << 52);
}

// X of a matrix whose norm is below eps is small, and its planes would hold few of its bits.  It is held times 2^q more, such that Z = 2^q X
// has a norm between 1/4 and 1.  A step takes Z to 2^(q' - q) (a Z + (b 4^-q + c 16^-q Z Z^T) Z Z^T Z), where q' is q less `growth`, 0 at the
// least, and 2^growth at least |p(s) / s| of the polynomial p: so Z's singular values stay within what X's are within.
// (2^100: there X reaches the smallest numbers of float32 itself.)
__device__ __forceinline__ int exponent_of(double v) { return static_cast<int>(__double_as_longlong(v) >> 52 & 0x7ff) - 1023; }
__device__ __forceinline__ int ortho_shift(double norm, double eps) {
    const int all = exponent_of(norm + eps), own = exponent_of(norm);  // (their difference is off by less than one)
    return all == 1024 || norm == 0. ? 0 : min(max(all - own - 1, 0), 100);
}
__device__ __forceinline__ float power_of_two(int n) {  // (0 below float32's normal numbers)
    return __uint_as_float(static_cast<uint32_t>(max(n + 127, 0)) << 23);
}

// 2^13 2^shift / norm as 2^up * factor, up a power that float32 holds and the factor
// near 1 where it can be: X's elements stay in range between.  A norm below 2^-160 is that of zeros and a smaller eps (the
// smallest number that is not zero is 2^-149): they stay zeros with any factor that float32 holds.  0: NaN.
// (Exponents as integers: a comparison in 64 bits by every warp of an SM costs what 16 in 32 bits do.)
struct OrthoScale {
    float power, factor;
    __device__ __forceinline__ OrthoScale(double norm, int shift) {
        if (__double_as_longlong(norm) != 0 && exponent_of(norm) < -160) norm = 0x1p-160;
        const double inv = 1. / norm;
        const int up = min(max(exponent_of(inv) + shift, -126), 126);
        power = power_of_two(up);
        factor = static_cast<float>(inv * __longlong_as_double(static_cast<long long>(1023 + shift - up) << 52)) * 8192.f;
    }
    __device__ __forceinline__ void split(const float (&v)[8], uint4& hi, uint4& lo) const {
        uint32_t h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = v[2 * j] * power * factor, y = v[2 * j + 1] * power * factor;
            const __half2 pair = __floats2half2_rn(x, y);
            h[j] = *reinterpret_cast<const uint32_t*>(&pair);
            l[j] = pair_from_f32<__half>(x - __low2float(pair), y - __high2float(pair));
        }
        hi = make_uint4(h[0], h[1], h[2], h[3]);
        lo = make_uint4(l[0], l[1], l[2], l[3]);
    }
};

}  // namespace gb300
