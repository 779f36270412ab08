// Routing of tokens to experts, and its gradient (include/sgemm_routing.h).
//
// Two forms.  A warp takes a token (route_kernel): lane l holds the scores of experts l * NPL
// .. l * NPL + NPL - 1, so that a row comes in with wide loads, a lane's experts are
// neighbours (groups span whole lanes) and the lowest of equal experts is the
// lowest lane's.  Scores are compared as unsigned keys in their order, 0 for
// an expert out of service: the warp's largest is then one redux instruction,
// and k of them with the lane's own largest kept up to date make the choice.
// Or four lanes take a token (route_quads_kernel), up to 8 of 256 experts: what the other
// form does once a warp for a token is done for eight at a time.
//
// What the choice is by.  Without a bias, or with one that is the same for all (and
// with group_best = 1), both scores grow with the logit, so logits are compared.  Otherwise float32 scores
// decide where they are further apart than their errors.  First with keys that
// hold the expert and 22 bits of the value (choose_packed); a token where two that
// decide are too near for that goes through keys of 32 bits, and scores that are
// too near for those are computed in 64 (choose_again), so that no rounding moves
// a choice.
//
// Places.  A CTA takes tokens 32 (or 16) at a time and sets a bit a token in a word of
// each chosen expert (an OR: its order does not matter); a choice's place
// among the expert's rows in this CTA is then the number of bits below its own
// plus those of the steps before.  The CTAs of a cluster add up their counts
// through distributed shared memory.  Up to 256 (512) tokens are one cluster, which
// then knows all; else the clusters' counts go to a table, and place_kernel adds
// up those of the clusters and of the experts before.
//
// Bound by instructions, not by bytes (16384 x 256 bf16: 10 MB, 1.5 us): about 1000 of
// a warp a token for scores, grid, sort and k rounds, 420 with four lanes a token, whose warps also wait for the
// instructions themselves (50 KB without a loop);
// for a few tokens by latency.  Measured on GB300 (replayed from a CUDA graph): 16384 tokens, 8 of 256
// experts, sigmoid, bias, 4 of 8 groups 28 to 32 us (43 with a warp a token; 22 where no scores lie so near one another
// that choose_again decides, which all wait for; with a bias of zeros, where equal bf16 logits are many, 48, with all logits equal
// 194, and 334 with all within 1e-6 of one another: groups by their best two are then summed in 64 bits for every token), by softmax alone 19 us
// (22), 64 tokens of the former 6.5 us; 65536 tokens, 6 of 64 27 us; one token, 4 of 64 3.4 us.  (ptxas: 76 to 92 bytes of spills with a
// warp a token and 128 or 256 experts, 128 to 136 in choose_again; none in the other kernels.)  What carried it:
// keys that hold their expert (51 -> 26 us by softmax), no
// division and no float64 but for the contested values (60 -> 47 us), clusters instead of a
// second launch (64 tokens 16 -> 6 us), four lanes a token (43 -> 37 us), choose_again's values in registers (37 -> 28 us).
#include <algorithm>
#include <type_traits>

#include "../../include/sgemm_routing.h"
#include "experts_groups.cuh"
#include "ptx.cuh"
#include "routing.h"

namespace gb300 {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRouteThreads = 32 * kRouteWarps;

// ------------------------------------------------------------------ keys

// Floating values as unsigned integers in their order: larger value, larger
// key; NaN the largest, no key 0, one key for both zeros.
template <typename V>
struct Keys;
template <>
struct Keys<float> {
    using Key = uint32_t;
    static __device__ __forceinline__ Key of(float v) {
        const uint32_t b = __float_as_uint(v + 0.f);
        return v != v ? ~0u : b ^ (b >> 31 ? ~0u : 0x80000000u);
    }
    static __device__ __forceinline__ float value(Key k) {
        return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : ~0u));  // (the key of NaN gives a NaN)
    }
    static __device__ __forceinline__ Key most(Key k) { return __reduce_max_sync(kAll, k); }
};
template <>
struct Keys<double> {
    using Key = unsigned long long;
    static __device__ __forceinline__ Key of(double v) {
        const Key b = static_cast<Key>(__double_as_longlong(v + 0.));
        return v != v ? ~0ull : b ^ (b >> 63 ? ~0ull : 1ull << 63);
    }
    static __device__ __forceinline__ double value(Key k) {
        return __longlong_as_double(static_cast<long long>(k ^ (k >> 63 ? 1ull << 63 : ~0ull)));
    }
    static __device__ __forceinline__ Key most(Key k) {
        const uint32_t hi = static_cast<uint32_t>(k >> 32), top = __reduce_max_sync(kAll, hi);
        const uint32_t lo = __reduce_max_sync(kAll, hi == top ? static_cast<uint32_t>(k) : 0u);
        return static_cast<Key>(top) << 32 | lo;
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d /= 2) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int d = 16; d; d /= 2) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
// (a NaN is passed over)
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d; d /= 2) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
}

// ------------------------------------------------------------------ rows

// A lane's values of a row of E: elements `first` ..., -inf past the row's end.
template <int NPL, typename T>
__device__ __forceinline__ void load_row(const T* row, int first, int E, bool vec, float (&v)[NPL]) {
    constexpr int kBytes = NPL * static_cast<int>(sizeof(T)), kWord = kBytes < 16 ? kBytes : 16;
    if (kWord >= 4 && vec && first + NPL <= E) {
        alignas(16) T x[NPL];
#pragma unroll
        for (int i = 0; i < kBytes; i += kWord) {
            const char* at = reinterpret_cast<const char*>(row + first) + i;
            char* to = reinterpret_cast<char*>(x) + i;
            if constexpr (kWord == 16)
                *reinterpret_cast<uint4*>(to) = __ldg(reinterpret_cast<const uint4*>(at));
            else if constexpr (kWord == 8)
                *reinterpret_cast<uint2*>(to) = __ldg(reinterpret_cast<const uint2*>(at));
            else if constexpr (kWord == 4)
                *reinterpret_cast<uint32_t*>(to) = __ldg(reinterpret_cast<const uint32_t*>(at));
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) v[i] = to_f32(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) v[i] = first + i < E ? to_f32(row[first + i]) : -INFINITY;
    }
}

// ------------------------------------------------------------------ the choice

// The two largest of four keys, (a >= b) and (c >= d), to a and b.
template <typename Key>
__device__ __forceinline__ void merge_two(Key& a, Key& b, Key c, Key d) {
    const Key low = min(a, c);
    a = max(a, c);
    b = max(low, max(b, d));
}

// The two best keys of group g, in lane g (0: none): any groups.
template <int NPL, typename Key>
__device__ __forceinline__ void group_best(const Key (&key)[NPL], const RouteParams& p, Key& a, Key& b) {
    const int lane = threadIdx.x & 31, first = lane * NPL, size = p.group_size;
    a = b = 0;
    for (int g = 0; g < p.groups; ++g) {
        Key c = 0, d = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = first + i - g * size;
            if (e >= 0 && e < size) merge_two(c, d, key[i], Key{0});
        }
#pragma unroll
        for (int s = 1; s < 32; s *= 2) merge_two(c, d, __shfl_xor_sync(kAll, c, s), __shfl_xor_sync(kAll, d, s));
        if (lane == g) a = c, b = d;
    }
}

// Keys of the groups that are not kept become 0.
template <int NPL, typename Key>
__device__ __forceinline__ void keep_groups(Key (&key)[NPL], const RouteParams& p, unsigned kept) {
    const int first = (threadIdx.x & 31) * NPL, size = p.group_size;
    int g = first / size, rest = first - g * size;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        if (g >= p.groups || !(kept >> g & 1)) key[i] = 0;
        if (++rest == size) rest = 0, ++g;
    }
}

// e^x to 2^-22 and 2^-24 |x|, relative: the rounding of x log2(e), and the instruction's 2 units.
__device__ __forceinline__ float fast_exp(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
    return y;
}
__device__ __forceinline__ float fast_reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (a NaN wins)
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// A row's largest logit (NaN passed over) and the sum of exp(l - top).
template <int NPL>
__device__ __forceinline__ void softmax_sums(const float (&l)[NPL], float& top, float& sum) {
    top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) top = fmaxf(top, l[i]);
    top = warp_max(top);
#pragma unroll
    for (int i = 0; i < NPL; ++i) sum += l[i] == -INFINITY ? 0.f : fast_exp(l[i] - top);
    sum = warp_sum(sum);
}

// `one_bias`: there is none, or it is the same finite number for all experts.
__device__ __forceinline__ bool chosen_by_logit(const RouteParams& p, bool one_bias) {
    return one_bias && (p.groups == 1 || p.group_best == 1);
}

// What an expert is chosen by where that is not the logit: c = score + bias, in
// float32, -inf out of service.  inv: 1 / sum.
__device__ __forceinline__ float choice_value(const RouteParams& p, float l, float bias, float top, float inv) {
    const float s = p.sigmoid ? fast_reciprocal(1.f + fast_exp(-l)) : fast_exp(l - top) * inv;
    return l == -INFINITY ? -INFINITY : s + bias;
}

// How far apart two of them have to be for their order to be certain; `size`: at
// least their magnitude.  Softmax: exp(l - top) is off by |l - top| 2^-23 (the
// roundings of the difference and of its multiple) and 2^-22; times exp(l - top), the
// former is largest at |l - top| = 1; the sum by as much, with 10 roundings and the mean of
// |l - top| over the softmax, below log 1024 = 7: in all below 2^-19 of the
// largest score, 1 / sum.  Sigmoid: s (1 - s) times the exponential's error, |l| s (1 - s) < 1/4,
// and two roundings: below 2^-21.  Then half a unit of the sum with the bias.
__device__ __forceinline__ float choice_error(const RouteParams& p, float size, float sum) {
    return 0x1p-22f * size + (p.sigmoid ? 0x1p-20f : 0x1p-18f * fast_reciprocal(sum));
}

// Loops over a lane's values are unrolled as long as registers hold these.
template <int NPL>
constexpr int kUnrolled = NPL <= 8 ? NPL : 1;

// The largest key's place: (lane, number) with the lowest expert.  Whole warp; 0 if there is none.
template <int NPL, typename V>
__device__ __forceinline__ typename Keys<V>::Key largest(const typename Keys<V>::Key (&key)[NPL], int& e) {
    typename Keys<V>::Key m = key[0];
    int at = 0;
#pragma unroll kUnrolled<NPL>
    for (int i = 1; i < NPL; ++i)
        if (key[i] > m) m = key[i], at = i;
    const auto best = Keys<V>::most(m);
    const int from = __ffs(__ballot_sync(kAll, m == best)) - 1;
    e = __shfl_sync(kAll, static_cast<int>(threadIdx.x & 31) * NPL + at, from);
    return best;
}

__device__ __noinline__ double exp64(double x) { return exp(x); }

// The choice with keys of 32 bits.  Where those that decide are within their
// errors of one another, these alone are compared again: by their logits if they
// have one bias (a bias of zeros, or equal scores of which a token of
// padding has many), else computed in 64 bits.
// Few tokens come here, and the rest wait for them: so little is computed in 64
// bits (2 lanes a cycle of an SM), in one place (instructions that
// nobody has fetched before: 25 us for the first token of a prompt with the loops around them unrolled).
template <int NPL, typename T>
__device__ __noinline__ int choose_again(const RouteParams& p, const T* row, bool by_logit, float top, float sum) {
    using K = Keys<float>;
    const int lane = threadIdx.x & 31, first = lane * NPL;
    float l[NPL], bias[NPL], size = 0.f, near = 0.f;
    uint32_t key[NPL];
#pragma unroll kUnrolled<NPL>
    for (int i = 0; i < NPL; ++i) {
        const bool there = first + i < p.E;
        l[i] = there ? to_f32(row[first + i]) : -INFINITY;
        bias[i] = there && p.bias ? p.bias[first + i] : 0.f;
    }
    const float inv = fast_reciprocal(sum);
#pragma unroll kUnrolled<NPL>
    for (int i = 0; i < NPL; ++i) {
        float c = l[i];
        if (!by_logit) {
            c = choice_value(p, c, bias[i], top, inv);
            if (fabsf(c) < INFINITY) size = fmaxf(size, fabsf(c));
        }
        key[i] = c == -INFINITY ? 0u : K::of(c);
    }
    if (!by_logit) near = choice_error(p, warp_max(size), sum);  // (logits are exact)
    double all = 0;  // the softmax's sum, once it is needed
    // use(i, 64-bit key) for the lane's values whose bit is set in `some`, one after another; one that is as the one before
    // is not computed again.
    auto evaluate = [&](uint32_t some, auto use) {
        const double less = p.sigmoid ? 0. : static_cast<double>(top);
        if (!p.sigmoid && all == 0) {
#pragma unroll 1
            for (int i = 0; i < NPL; ++i) all += first + i < p.E ? exp64(to_f32(row[first + i]) - less) : 0.;
            all = warp_sum(all);
        }
        float before = NAN, before_bias = 0.f;
        unsigned long long value = 0;
        for (; __any_sync(kAll, some); some &= some - 1) {
            if (some) {
                const int i = __ffs(some) - 1;
                const float logit = to_f32(row[first + i]), b = p.bias ? p.bias[first + i] : 0.f;
                if (!(logit == before && b == before_bias)) {
                    const double x = logit - less, y = exp64(p.sigmoid ? -x : x);
                    value = Keys<double>::of((p.sigmoid ? 1. / (1. + y) : y / all) + b);
                    before = logit, before_bias = b;
                }
                use(i, value);
            }
        }
    };
    if (p.groups > 1) {
        uint32_t a, b;
        group_best<NPL>(key, p, a, b);
        const bool there = lane < p.groups && a;
        float score = 0.f;
        // (half the sum of two: that of finite values is finite.  Not half of one: logits may be the smallest numbers)
        if (there) score = p.group_best == 2 ? 0.5f * K::value(a) + (b ? 0.5f * K::value(b) : 0.f) : K::value(a);
        const uint32_t rank = there ? K::of(score) : 0u;
        // Surely among the best: fewer than top_groups may be better.  Surely not: as many are.
        int may = 0, are = 0;
        for (int g = 0; g < p.groups; ++g) {
            const uint32_t other = __shfl_sync(kAll, rank, g);
            const float v = __shfl_sync(kAll, score, g);
            if (g == lane || !other) continue;
            const bool close = near > 0.f && fabsf(score) < INFINITY && fabsf(v) < INFINITY && fabsf(v - score) <= near;
            const bool better = other > rank || (other == rank && g < lane);
            may += close || better;
            are += !close && better;
        }
        unsigned kept = __ballot_sync(kAll, there && may < p.top_groups);
        const unsigned open = __ballot_sync(kAll, there && may >= p.top_groups && are < p.top_groups);
        if (open) {
            // The open groups' scores in 64 bits, from those of their values that may be among the best two.
            const int size = p.group_size;
            const float second = b ? K::value(b) : -INFINITY;
            uint32_t some = 0;
            unsigned long long exact[NPL] = {}, best, next;
            int g = first / size, rest = first - g * size;
#pragma unroll kUnrolled<NPL>
            for (int i = 0; i < NPL; ++i) {
                const float from = __shfl_sync(kAll, p.group_best == 2 ? second : there ? K::value(a) : 0.f, g) - near;
                if (key[i] && g < 32 && (open >> g & 1) && !(K::value(key[i]) < from)) some |= 1u << i;
                if (++rest == size) rest = 0, ++g;
            }
            evaluate(some, [&](int at, unsigned long long x) {
#pragma unroll kUnrolled<NPL>
                for (int i = 0; i < NPL; ++i)
                    if (i == at) exact[i] = x;
            });
            group_best<NPL>(exact, p, best, next);
            unsigned long long value = 0;
            if (open >> lane & 1) {
                double v = Keys<double>::value(best);
                if (p.group_best == 2 && next) v += Keys<double>::value(next);
                value = Keys<double>::of(v);
            }
            for (int left = p.top_groups - __popc(kept); left > 0; --left) {
                const unsigned long long most = Keys<double>::most(value);
                if (most == 0) break;
                const int from = __ffs(__ballot_sync(kAll, value == most)) - 1;
                kept |= 1u << from;
                if (lane == from) value = 0;
            }
        }
        keep_groups<NPL>(key, p, kept);
    }
    int mine = -1;
    for (int j = 0; j < p.k; ++j) {
        int e;
        const uint32_t best = largest<NPL, float>(key, e);
        if (best == 0) break;
        const float v = K::value(best);
        if (near > 0.f && fabsf(v) < INFINITY) {
            const uint32_t from = K::of(v - near);
            uint32_t some = 0;
#pragma unroll kUnrolled<NPL>
            for (int i = 0; i < NPL; ++i)
                if (key[i] >= from) some |= 1u << i;
            if (__reduce_add_sync(kAll, __popc(some)) > 1) {
                const float one = p.bias ? p.bias[e] : 0.f;
                bool other = false;
                uint32_t logit[NPL];
#pragma unroll kUnrolled<NPL>
                for (int i = 0; i < NPL; ++i) {
                    logit[i] = some >> i & 1 ? K::of(l[i]) : 0u;
                    other |= (some >> i & 1) && bias[i] != one;
                }
                if (__any_sync(kAll, other)) {
                    unsigned long long top64 = 0;
                    int at = 0;
                    evaluate(some, [&](int i, unsigned long long x) {
                        if (x > top64) top64 = x, at = i;
                    });
                    const unsigned long long best64 = Keys<double>::most(top64);
                    e = __shfl_sync(kAll, first + at, __ffs(__ballot_sync(kAll, top64 == best64)) - 1);
                } else {
                    (void)largest<NPL, float>(logit, e);
                }
            }
        }
        if (lane == j) mine = e;
#pragma unroll kUnrolled<NPL>
        for (int i = 0; i < NPL; ++i)
            if (first + i == e) key[i] = 0;
    }
    return mine;
}

// Keys with their expert in them: 22 bits of the value, in its order, and 1023 - e
// below.  No two are alike, so that a maximum names its expert, and equal
// values go to the lowest.  Of a 16-bit logit the upper 22 bits of its key in
// float32 are all there is; other values are taken to a grid of 2^22 steps from
// the token's smallest to its largest.  Keys below 1024: out of service.
constexpr uint32_t kExpertBits = 1023;
constexpr int kExpertShift = 10;

// Exchanges that sort the lane's keys, the largest first (merge exchange, Batcher).
template <int NPL>
__device__ __forceinline__ void sort_lane(uint32_t (&key)[NPL]) {
#pragma unroll
    for (int p = 1; p < NPL; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < NPL; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < NPL && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t x = key[i + j], y = key[i + j + k];
                        key[i + j] = max(x, y);
                        key[i + j + k] = min(x, y);
                    }
}

// The choice with packed keys: lane j's result is the j-th expert, -1 where there
// is none.  exact: they hold all of the values; else `sure` is false where two
// that decide are not further apart than `gap` steps of the grid (the scores of
// groups: `group_gap`).
template <int NPL>
__device__ __forceinline__ int choose_packed(uint32_t (&key)[NPL], const RouteParams& p, bool exact, uint32_t gap,
                                             uint32_t group_gap, bool& sure) {
    const int lane = threadIdx.x & 31;
    constexpr bool SORTED = NPL <= 8;
    bool close = false;
    auto most = [](uint32_t k) { return __reduce_max_sync(kAll, k); };
    // Groups that are a power of two of whole lanes, 2^shift of them, or no groups.
    const bool whole = SORTED && p.group_lanes >= 0;
    const int shift = max(p.group_lanes, 0), lanes = 1 << shift;
    if constexpr (SORTED) {
        if (whole) sort_lane(key);
    }
    if (p.groups > 1) {
        uint32_t a, b;
        if (whole) {
            a = key[0], b = NPL > 1 ? key[NPL > 1 ? 1 : 0] : 0u;
            for (int d = 1; d < lanes; d *= 2) merge_two(a, b, __shfl_xor_sync(kAll, a, d), __shfl_xor_sync(kAll, b, d));
            const int from = (lane << shift) & 31;
            a = __shfl_sync(kAll, a, from);
            b = __shfl_sync(kAll, b, from);
        } else {
            group_best<NPL>(key, p, a, b);
        }
        a >>= kExpertShift;
        b >>= kExpertShift;
        uint32_t score = lane < p.groups ? a : 0u;
        if (p.group_best == 2) {
            // (a sum of two and a single value are not on one grid)
            const unsigned one = __ballot_sync(kAll, score != 0 && b == 0), two = __ballot_sync(kAll, score != 0 && b != 0);
            close = one && two;
            if (score) score += b;
        }
        unsigned kept = 0;
        uint32_t last = ~0u;
        for (int i = 0; i < p.top_groups; ++i) {
            const uint32_t best = most(score);
            const unsigned who = __ballot_sync(kAll, score == best);
            const unsigned bit = who & (0u - who);  // the lowest
            kept |= best ? bit : 0u;
            if (bit >> lane & 1) score = 0;
            last = best;
        }
        const uint32_t next = most(score);
        close |= next && last - next <= group_gap;
        if (whole) {
            if (!(kept >> (lane >> shift) & 1)) {
#pragma unroll
                for (int i = 0; i < NPL; ++i) key[i] = 0;
            }
        } else {
            keep_groups<NPL>(key, p, kept);
        }
    }
    uint32_t m = key[0];
    if constexpr (SORTED) {
        if (!whole) sort_lane(key);
        m = key[0];
    } else {
#pragma unroll
        for (int i = 1; i < NPL; ++i) m = max(m, key[i]);
    }
    uint32_t before = ~0u;
    int mine = -1;
    for (int j = exact ? 1 : 0; j <= p.k; ++j) {  // (one more than wanted, to see how near it is)
        const uint32_t best = most(m);
        close |= j > 0 && best > kExpertBits && (before >> kExpertShift) - (best >> kExpertShift) <= gap;
        if (lane == (exact ? j - 1 : j)) mine = best > kExpertBits ? static_cast<int>(kExpertBits - (best & kExpertBits)) : -1;
        before = best;
        if constexpr (SORTED) {
            const bool pop = m == best;
#pragma unroll
            for (int i = 0; i + 1 < NPL; ++i) key[i] = pop ? key[i + 1] : key[i];
            key[NPL - 1] = pop ? 0u : key[NPL - 1];
            m = key[0];
        } else if (m == best) {
            m = 0;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                key[i] = key[i] == best ? 0u : key[i];
                m = max(m, key[i]);
            }
        }
    }
    sure = exact || !close;
    return lane < p.k ? mine : -1;
}

// The largest of the lane's values (NaN before all) and the smallest of those in service.
template <int NPL>
__device__ __forceinline__ void range_of(const float (&c)[NPL], float& high, float& low) {
    high = -INFINITY, low = INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        high = max_nan(high, c[i]);
        low = fminf(low, c[i] == -INFINITY ? INFINITY : c[i]);
    }
}

// Keys on a grid from the smallest value of a token to its largest, `range` in all.  A value's place is off
// by less than a step, and places never change their order.  There is no grid for values that are all alike, or not finite.
__device__ __forceinline__ bool on_grid(float range) { return range > 0x1p-60f && range < 0x1p60f; }
__device__ __forceinline__ float grid_scale(float range) { return 4194280.f * fast_reciprocal(range); }  // 2^22 less 24
template <int NPL>
__device__ __forceinline__ void place_on_grid(const float (&c)[NPL], float low, float scale, int first, uint32_t (&key)[NPL]) {
    // The place is the mantissa of a number from 2^23 on, whose exponent the shift drops (as it drops all of -inf).
    const uint32_t e0 = kExpertBits - first;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        key[i] = (__float_as_uint(fmaf(c[i] - low, scale, 8388612.f)) << kExpertShift) + (e0 - static_cast<uint32_t>(i));
}

// A warp's keys on the grid; false where there is none.
template <int NPL>
__device__ __forceinline__ bool grid_keys(const float (&c)[NPL], uint32_t (&key)[NPL], float& low, float& high,
                                          float& scale) {
    using K = Keys<float>;
    range_of(c, high, low);
    high = K::value(__reduce_max_sync(kAll, K::of(high)));
    low = K::value(__reduce_min_sync(kAll, K::of(low)));
    scale = grid_scale(high - low);
    place_on_grid(c, low, scale, (threadIdx.x & 31) * NPL, key);
    return on_grid(high - low);
}

// How many steps of the grid apart two scores have to be (a step more for each place's error), and two scores of groups.
// The grid has 2^22 steps however near a token's values are to one another: where their errors are larger than all of it, so is
// this (2^23 at most, and 2^24 for the sums of groups, which are below 2^23), and nothing is certain.
__device__ __forceinline__ float choice_steps(const RouteParams& p, float low, float high, float sum, float scale) {
    return fminf(choice_error(p, fmaxf(fabsf(low), fabsf(high)), sum) * scale, 0x1p23f);
}
__device__ __forceinline__ uint32_t choice_gap(float steps) { return static_cast<uint32_t>(steps + 2.1f); }
__device__ __forceinline__ uint32_t score_gap(const RouteParams& p, float steps) {
    return p.group_best == 2 ? static_cast<uint32_t>(2.f * steps + 4.1f) : choice_gap(steps);
}

// A token's experts, the j-th in lane j, from its logits (the lane's part); `bias`: the lane's, in shared memory.
template <int NPL, typename T>
__device__ __forceinline__ int choose_experts(const RouteParams& p, const float (&l)[NPL], bool by_logit, const float* bias,
                                              float top, float sum, bool& sure) {
    uint32_t key[NPL];
    float low, high, scale;
    if (by_logit) {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const uint32_t e = (threadIdx.x & 31) * NPL + i;
                key[i] = l[i] == -INFINITY ? 0u : (Keys<float>::of(l[i]) & ~kExpertBits) | (kExpertBits - e);
            }
            return choose_packed<NPL>(key, p, true, 0, 0, sure);
        } else {
            sure = grid_keys(l, key, low, high, scale);
            if (sure) return choose_packed<NPL>(key, p, false, 0, 0, sure);
            sure = high == -INFINITY;  // (nobody is in service)
            return -1;
        }
    }
    float c[NPL], b[NPL];
    if constexpr (NPL >= 4) {
#pragma unroll
        for (int i = 0; i < NPL; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(bias + i);
            b[i] = x.x, b[i + 1] = x.y, b[i + 2] = x.z, b[i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) b[i] = bias[i];
    }
    const float inv = fast_reciprocal(sum);
#pragma unroll
    for (int i = 0; i < NPL; ++i) c[i] = choice_value(p, l[i], b[i], top, inv);
    sure = grid_keys(c, key, low, high, scale);
    if (!sure) {
        sure = high == -INFINITY;  // (nobody is in service)
        return -1;
    }
    const float steps = choice_steps(p, low, high, sum, scale);
    return choose_packed<NPL>(key, p, false, choice_gap(steps), score_gap(p, steps), sure);
}

// The score of logit x, less the factor of `lead` that all of a token's have.
//
// sigmoid(l) = e^min(l, 0) / (1 + e^-|l|): with the largest chosen logit's
// e^min(l, 0) taken out, the renormalised ones are ratios of numbers near 1
// however small the scores are.
// Softmax: an expert that its bias had chosen may lie far below the largest logit, where the rounding of the difference alone, up to
// 2^-18 from 64 on, is as large as the weight's error may be: it is added back, e^(d + r) = e^d (1 + r).
__device__ __forceinline__ float score_over(const RouteParams& p, float x, float lead, float sum) {
    if (p.sigmoid) {
        const float low = x > 0.f ? 0.f : x;
        return __fdividef(expf(low - (p.renormalize ? fminf(lead, 0.f) : 0.f)), 1.f + expf(-fabsf(x)));
    }
    if (sum != sum) return sum;  // (a NaN or +inf that was not chosen)
    const float d = x - lead, e = expf(d);
    if (!(d > -128.f)) return e;  // (0, or NaN)
    const float less = x - d;
    return fmaf(e, (x - (d + less)) + (less - lead), e);
}

// The weight of the lane's expert e (-1: none).
template <typename T>
__device__ __forceinline__ float weight_of(const RouteParams& p, const T* row, int e, float top, float sum) {
    const float x = e >= 0 ? to_f32(row[e]) : -INFINITY;
    const float lead = p.renormalize ? warp_max(x) : top;
    float s = e < 0 ? 0.f : score_over(p, x, lead, sum);
    if (p.renormalize) sum = warp_sum(s);
    return e < 0 ? 0.f : p.sigmoid && !p.renormalize ? p.scale * s : p.scale * s * fast_reciprocal(sum);
}

// Exclusive sums of count[0 .. E - 1] (at most two a thread) to base, and
// offsets if `out`.  Whole CTA; `scratch` of a word a warp.
__device__ __forceinline__ void exclusive_sums(const int* count, int E, int* base, int* out, int* scratch) {
    const int i = 2 * threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int a = i < E ? count[i] : 0, b = i + 1 < E ? count[i + 1] : 0;
    int sum = a + b;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(kAll, sum, d);
        if (lane >= d) sum += v;
    }
    if (lane == 31) scratch[warp] = sum;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += scratch[w];
    const int from = before + sum - a - b;
    if (i < E) base[i] = from;
    if (i + 1 < E) base[i + 1] = from + a;
    if (out) {
        if (i < E) out[i] = from;
        if (i + 1 < E) out[i + 1] = from + a;
        if (i + 1 == E || i + 2 == E) out[E] = from + a + b;
    }
    __syncthreads();
}

// The CTAs of a cluster add up their counts: `before` those of the CTAs before this one, `sums` those of all, which
// also go to p.counts.
__device__ __forceinline__ void cluster_counts(const RouteParams& p, const int* count, int* before, int* sums) {
    const int of = static_cast<int>(cluster_ctarank());
    cluster_sync_all();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        const uint32_t at = smem_addr(count + e);
        int sum = 0, sum_before = 0;
#pragma unroll 4
        for (int q = 0; q < p.width; ++q) {
            if (q == of) sum_before = sum;
            sum += ld_shared_cluster_s32(map_shared_rank(at, q));
        }
        before[e] = sum_before;
        sums[e] = sum;
        if (p.counts && of == 0) p.counts[static_cast<long long>(blockIdx.x / p.width) * p.E + e] = sum;
    }
    cluster_sync_all();  // (nobody reads this CTA's counts after this)
}

// One cluster did it all: what comes before a CTA's choices of an expert among all, to `before`, and the boundaries.
__device__ __forceinline__ void finish_counts(const RouteParams& p, int* base, int* before, const int* sums, int* scratch) {
    exclusive_sums(sums, p.E, base, blockIdx.x == 0 ? p.offsets : nullptr, scratch);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) before[e] += base[e];
    __syncthreads();
}

// The CTAs of a cluster (p.width) add up their counts of each expert's choices
// through distributed shared memory.  With p.counts there are several clusters,
// which leave their sums there for place_kernel; else the one finishes the places.
template <int NPL, typename T>
__global__ void __launch_bounds__(kRouteThreads, NPL <= 8 ? 2 : 1) route_kernel(const RouteParams p) {
    extern __shared__ __align__(16) int shared[];
    float* const bias = reinterpret_cast<float*>(shared);  // 32 * NPL
    int* const mask = shared + 32 * NPL;                   // E: this step's tokens
    int* const count = mask + p.E;                         // E: choices of the steps before
    int* const before = count + p.E;    // E: of the cluster's CTAs before this one, then all that come before
    int* const scratch = before + p.E;  // a word a warp
    grid_dependency_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) mask[e] = count[e] = 0;
    const float first_bias = p.bias ? __ldg(p.bias) : 0.f;
    bool same = fabsf(first_bias) < INFINITY;
    for (int e = threadIdx.x; e < 32 * NPL; e += kRouteThreads) {
        const float b = p.bias && e < p.E ? __ldg(p.bias + e) : first_bias;
        same &= b == first_bias;
        bias[e] = b;
    }
    const bool by_logit = chosen_by_logit(p, __syncthreads_and(same));
    constexpr int kTokens = 2;  // of a warp in a step, at most: with 16 warps, a bit each
    static_assert(kTokens * kRouteWarps <= 32, "a bit a token");
    const bool sums = !p.sigmoid && (!p.renormalize || !by_logit);
    const long long begin = static_cast<long long>(blockIdx.x) * p.per, end = min(static_cast<long long>(p.T), begin + p.per);
    int mine[kTokens] = {}, rank[kTokens] = {};  // of the last step
    for (int step = 0; step < p.steps; ++step) {
        const long long t0 = begin + step * p.step + warp;
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            const long long t = t0 + i * kRouteWarps;
            mine[i] = -1;
            if (t < end && i * kRouteWarps < p.step) {
                const T* const row = static_cast<const T*>(p.logits) + t * p.ld;
                float top = 0.f, sum = 0.f;
                bool sure;
                int e;
                {
                    float l[NPL];
                    load_row<NPL>(row, lane * NPL, p.E, p.vec, l);
                    if (sums) softmax_sums(l, top, sum);
                    e = choose_experts<NPL, T>(p, l, by_logit, bias + lane * NPL, top, sum, sure);
                }
                if (!sure) e = choose_again<NPL>(p, row, by_logit, top, sum);
                const float w = weight_of(p, row, e, top, sum);
                if (lane < p.k) {
                    p.experts[t * p.k + lane] = e;
                    p.weights[t * p.k + lane] = w;
                    if (e >= 0) atomicOr(mask + e, 1 << (warp + i * kRouteWarps));
                }
                mine[i] = e;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            const long long t = t0 + i * kRouteWarps;
            const unsigned below = (1u << (warp + i * kRouteWarps)) - 1;
            rank[i] = mine[i] < 0 ? -1 : count[mine[i]] + __popc(mask[mine[i]] & below);
            if (step + 1 < p.steps && t < end && i * kRouteWarps < p.step && lane < p.k) p.slots[t * p.k + lane] = rank[i];
        }
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
            count[e] += __popc(mask[e]);
            mask[e] = 0;
        }
        __syncthreads();
    }
    cluster_counts(p, count, before, mask);
    if (!p.counts) finish_counts(p, count, before, mask, scratch);
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const long long t = begin + (p.steps - 1) * p.step + warp + i * kRouteWarps;
        if (t < end && i * kRouteWarps < p.step && lane < p.k)
            p.slots[t * p.k + lane] = mine[i] < 0 ? -1 : rank[i] + before[mine[i]];
    }
    if (p.steps > 1) {  // the steps before the last, whose places are in memory
        const long long from = begin * p.k, to = min(end, begin + (p.steps - 1) * p.step) * p.k;
        for (long long i = from + threadIdx.x; i < to; i += kRouteThreads) {
            const int e = p.experts[i];
            if (e >= 0) p.slots[i] += before[e];
        }
    }
}

// ------------------------------------------------------------------ many tokens
//
// Four lanes a token, N = 16, 32 or 64 neighbouring experts a lane, the choice the
// same as choose_packed's.  What a warp does once for a token above (a maximum of all lanes for each choice and
// each group, the weights), it does here once for eight.  A lane's keys are sorted eight
// at a time (19 exchanges) and merged to the best eight; then two merges across the four.  Of what a merge drops the
// largest is kept, to see how near the ninth is.
constexpr int kQuadWarps = 4, kQuadThreads = 32 * kQuadWarps;
static_assert(8 * kQuadWarps == kQuadStep, "a bit a token");

// The best eight of two sorted eights to `a`, sorted; `next`: the largest that is dropped.
__device__ __forceinline__ void merge_best(uint32_t (&a)[8], const uint32_t (&b)[8], uint32_t& next) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        next = max(next, min(a[i], b[7 - i]));
        a[i] = max(a[i], b[7 - i]);
    }
#pragma unroll
    for (int d = 4; d; d /= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) {
                const uint32_t x = a[i], y = a[i + d];
                a[i] = max(x, y);
                a[i + d] = min(x, y);
            }
}

// Over the four lanes of a token.
template <typename V, typename F>
__device__ __forceinline__ V over_quad(V v, F f) {
    v = f(v, __shfl_xor_sync(kAll, v, 1));
    return f(v, __shfl_xor_sync(kAll, v, 2));
}

// choose_packed of four lanes: their keys to the best eight, sorted, in `best`.  Groups are powers of two from 8 on.
// False where it is not certain which these are; bit j of `near` where it is not that the j-th is behind the one before.
template <int N>
__device__ __forceinline__ bool choose_quad(uint32_t (&key)[N], const RouteParams& p, uint32_t gap, uint32_t group_gap,
                                            uint32_t (&best)[8], uint32_t& near) {
    constexpr int B = N / 8;  // blocks of eight keys
    const int block = (threadIdx.x & 3) * B;
    const auto most = [](uint32_t x, uint32_t y) { return max(x, y); };
    bool close = false;
    if (p.groups > 1) {
        const int blocks = p.group_size >> 3, shift = 31 - __clz(blocks);
        uint32_t a[B], b[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            a[j] = b[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) merge_two(a[j], b[j], key[8 * j + i], 0u);
        }
        // A group's first block gets what the others have: those of a lane, and of the next (a group is half of all experts at most).
#pragma unroll
        for (int w = 1; w < B; w *= 2)
            if (blocks > w) {
#pragma unroll
                for (int j = 0; j + w < B; j += 2 * w) merge_two(a[j], b[j], a[j + w], b[j + w]);
            }
        if (blocks > B) merge_two(a[0], b[0], __shfl_xor_sync(kAll, a[0], 1), __shfl_xor_sync(kAll, b[0], 1));
        // Scores with their group in them, as keys hold their expert.
        uint32_t score[B];
        bool one = false, two = false;
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const bool first = ((block + j) & (blocks - 1)) == 0;
            uint32_t v = first ? a[j] >> kExpertShift : 0u;
            const uint32_t second = p.group_best == 2 ? b[j] >> kExpertShift : 0u;
            one |= v && !second;
            two |= v && second;
            if (v) v += second;
            score[j] = v ? v << 5 | (31 - ((block + j) >> shift)) : 0u;
        }
        // (a sum of two and a single value are not on one grid)
        const unsigned ones = __ballot_sync(kAll, one), twos = __ballot_sync(kAll, two);
        const int quad = threadIdx.x & 28;
        close = (ones >> quad & 15) && (twos >> quad & 15);
        unsigned kept = 0;
        uint32_t last = ~0u;
        for (int i = 0; i <= p.top_groups; ++i) {
            uint32_t m = score[0];
#pragma unroll
            for (int j = 1; j < B; ++j) m = max(m, score[j]);
            m = over_quad(m, most);
            if (i == p.top_groups) {
                close |= m && last - (m >> 5) <= group_gap;
            } else {
                kept |= m ? 1u << (31 - (m & 31)) : 0u;
                last = m >> 5;
#pragma unroll
                for (int j = 0; j < B; ++j) score[j] = score[j] == m ? 0u : score[j];
            }
        }
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (!(kept >> ((block + j) >> shift & 31) & 1)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) key[8 * j + i] = 0;
            }
    }
    uint32_t next = 0;
#pragma unroll
    for (int j = 0; j < B; ++j) {
        uint32_t some[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) some[i] = key[8 * j + i];
        sort_lane(some);
        if (j == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) best[i] = some[i];
        } else {
            merge_best(best, some, next);
        }
    }
#pragma unroll
    for (int d = 1; d <= 2; d *= 2) {
        uint32_t other[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(kAll, best[i], d);
        next = max(next, __shfl_xor_sync(kAll, next, d));
        merge_best(best, other, next);
    }
#pragma unroll
    for (int j = 1; j <= 8; ++j) {
        const uint32_t here = j < 8 ? best[j & 7] : next;
        const bool two = here > kExpertBits && (best[j - 1] >> kExpertShift) - (here >> kExpertShift) <= gap;
        close |= j == p.k && two;
        near |= j < p.k && two ? 1u << j : 0u;
    }
    return !close;
}

// As route_kernel, for k <= 8 and E <= 4 N.
template <int N, typename T>
__global__ void __launch_bounds__(kQuadThreads, 4) route_quads_kernel(const RouteParams p) {
    constexpr int kPitch = N + 4;  // (the four lanes' vectors of the bias from other banks)
    extern __shared__ __align__(16) int shared[];
    float* const bias = reinterpret_cast<float*>(shared);  // 4 kPitch
    int* const mask = shared + 4 * kPitch;                 // E each, as route_kernel's
    int* const count = mask + p.E;
    int* const before = count + p.E;
    int* const scratch = before + p.E;  // a word a warp
    grid_dependency_launch();
    const int lane = threadIdx.x & 31, q = lane & 3, first = q * N;
    for (int e = threadIdx.x; e < p.E; e += kQuadThreads) mask[e] = count[e] = 0;
    const float first_bias = p.bias ? __ldg(p.bias) : 0.f;
    bool same = fabsf(first_bias) < INFINITY;
    for (int e = threadIdx.x; e < 4 * N; e += kQuadThreads) {
        const float b = p.bias && e < p.E ? __ldg(p.bias + e) : first_bias;
        same &= b == first_bias;
        bias[e / N * kPitch + e % N] = b;
    }
    const bool by_logit = chosen_by_logit(p, __syncthreads_and(same));
    const bool sums = !p.sigmoid && (!p.renormalize || !by_logit);
    const auto most = [](float x, float y) { return fmaxf(x, y); };
    const auto plus = [](float x, float y) { return x + y; };
    const long long begin = static_cast<long long>(blockIdx.x) * p.per, end = min(static_cast<long long>(p.T), begin + p.per);
    const int bit = threadIdx.x >> 2;
    int mine[2] = {-1, -1}, rank[2] = {-1, -1};  // choices q and q + 4 of the last step
    for (int step = 0; step < p.steps; ++step) {
        const long long t = begin + step * p.step + bit;
        const bool there = t < end;
        const T* const row = static_cast<const T*>(p.logits) + (there ? t : begin) * p.ld;
        float top = 0.f, sum = 0.f, low = 0.f, high = 0.f;
        bool sure;
        uint32_t near = 0;
        {
            float v[N];
            if (there) {
                load_row<N>(row, first, p.E, p.vec, v);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = -INFINITY;
            }
            if (sums) {
                top = -INFINITY;
#pragma unroll
                for (int i = 0; i < N; ++i) top = fmaxf(top, v[i]);
                top = over_quad(top, most);
                float part[8] = {};  // (few roundings; see choice_error)
#pragma unroll
                for (int i = 0; i < N; ++i) part[i % 8] += v[i] == -INFINITY ? 0.f : fast_exp(v[i] - top);
#pragma unroll
                for (int d = 4; d; d /= 2)
#pragma unroll
                    for (int i = 0; i < d; ++i) part[i] += part[i + d];
                sum = over_quad(part[0], plus);
            }
            uint32_t key[N], best[8], gap = 0, group_gap = 0;
            bool grid = true;
            if (sizeof(T) == 2 && by_logit) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    key[i] = v[i] == -INFINITY ? 0u : (Keys<float>::of(v[i]) & ~kExpertBits) | (kExpertBits - (first + i));
            } else {
                if (!by_logit) {
                    const float inv = fast_reciprocal(sum);
#pragma unroll
                    for (int i = 0; i < N; i += 4) {
                        const float4 x = *reinterpret_cast<const float4*>(bias + q * kPitch + i);
                        const float b[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u) v[i + u] = choice_value(p, v[i + u], b[u], top, inv);
                    }
                }
                high = -INFINITY, low = INFINITY;
                range_of(v, high, low);
                high = over_quad(high, [](float x, float y) { return max_nan(x, y); });
                low = over_quad(low, [](float x, float y) { return fminf(x, y); });
                const float scale = grid_scale(high - low);
                grid = on_grid(high - low);
                place_on_grid(v, low, scale, first, key);
                if (!by_logit) {
                    const float steps = choice_steps(p, low, high, sum, scale);
                    gap = choice_gap(steps), group_gap = score_gap(p, steps);
                }
            }
            sure = choose_quad(key, p, gap, group_gap, best, near);
            if (sizeof(T) == 2 && by_logit) sure = true, near = 0;
            if (!grid) sure = high == -INFINITY, near = 0;  // (nobody is in service)
            // choices q and q + 4
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t x = q & 1 ? best[4 * i + 1] : best[4 * i], y = q & 1 ? best[4 * i + 3] : best[4 * i + 2];
                const uint32_t b = q & 2 ? y : x;
                mine[i] = grid && b > kExpertBits && q + 4 * i < p.k ? static_cast<int>(kExpertBits - (b & kExpertBits)) : -1;
            }
        }
        // Choices that lie near one another are in order where their logits are, if they have one bias.
        if (__any_sync(kAll, near)) {
            const int behind = (lane & 28) | ((lane + 1) & 3);
            float l[2], b[2], next_l[2], next_b[2];
            int next_e[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[i] = mine[i] >= 0 ? to_f32(row[mine[i]]) : -INFINITY;
                b[i] = mine[i] >= 0 ? bias[mine[i] / N * kPitch + mine[i] % N] : 0.f;
                next_l[i] = __shfl_sync(kAll, l[i], behind);
                next_b[i] = __shfl_sync(kAll, b[i], behind);
                next_e[i] = __shfl_sync(kAll, mine[i], behind);
            }
            if (q == 3) next_l[0] = next_l[1], next_b[0] = next_b[1], next_e[0] = next_e[1];  // (the fifth is the first lane's)
            bool wrong = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool ordered = b[i] == next_b[i] && (l[i] > next_l[i] || (l[i] == next_l[i] && mine[i] < next_e[i]));
                wrong |= (near >> (q + 4 * i + 1) & 1) && !ordered;
            }
            if (__ballot_sync(kAll, wrong) >> (lane & 28) & 15) sure = false;
        }
        // The tokens that are not sure, one after another, by the whole warp.
        for (unsigned left = __ballot_sync(kAll, !sure && q == 0); left; left &= left - 1) {
            const int from = __ffs(left) - 1;
            const long long other = __shfl_sync(kAll, t, from);
            const int e = choose_again<N / 8>(p, static_cast<const T*>(p.logits) + other * p.ld, by_logit,
                                              __shfl_sync(kAll, top, from), __shfl_sync(kAll, sum, from));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int theirs = __shfl_sync(kAll, e, q + 4 * i);
                if ((lane & 28) == from) mine[i] = theirs;
            }
        }
        float x[2], s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) x[i] = mine[i] >= 0 ? to_f32(row[mine[i]]) : -INFINITY;
        const float lead = p.renormalize ? over_quad(fmaxf(x[0], x[1]), most) : top;
#pragma unroll
        for (int i = 0; i < 2; ++i) s[i] = mine[i] < 0 ? 0.f : score_over(p, x[i], lead, sum);
        if (p.renormalize) sum = over_quad(s[0] + s[1], plus);
        const float share = p.sigmoid && !p.renormalize ? 1.f : fast_reciprocal(sum);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = q + 4 * i;
            if (there && j < p.k) {
                p.experts[t * p.k + j] = mine[i];
                p.weights[t * p.k + j] = mine[i] < 0 ? 0.f : p.scale * s[i] * share;
                if (mine[i] >= 0) atomicOr(mask + mine[i], 1 << bit);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = q + 4 * i;
            rank[i] = mine[i] < 0 ? -1 : count[mine[i]] + __popc(mask[mine[i]] & ((1u << bit) - 1));
            if (step + 1 < p.steps && there && j < p.k) p.slots[t * p.k + j] = rank[i];
        }
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += kQuadThreads) {
            count[e] += __popc(mask[e]);
            mask[e] = 0;
        }
        __syncthreads();
    }
    cluster_counts(p, count, before, mask);
    if (!p.counts) finish_counts(p, count, before, mask, scratch);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const long long t = begin + (p.steps - 1) * p.step + bit;
        const int j = q + 4 * i;
        if (t < end && j < p.k) p.slots[t * p.k + j] = mine[i] < 0 ? -1 : rank[i] + before[mine[i]];
    }
    if (p.steps > 1) {  // the steps before the last, whose places are in memory
        const long long from = begin * p.k, to = min(end, begin + (p.steps - 1) * p.step) * p.k;
        for (long long i = from + threadIdx.x; i < to; i += kQuadThreads) {
            const int e = p.experts[i];
            if (e >= 0) p.slots[i] += before[e];
        }
    }
}

// Places within a cluster's rows of an expert to places among all rows.
__global__ void __launch_bounds__(kRouteThreads) place_kernel(const RouteParams p, int clusters) {
    extern __shared__ __align__(16) int shared[];
    int* const total = shared;
    int* const before = shared + p.E;
    int* const base = shared + 2 * p.E;
    int* const scratch = shared + 3 * p.E;
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) total[e] = before[e] = 0;
    __syncthreads();
    grid_dependency_wait();
    // (the first choices' experts on their way beside the counts)
    const long long per = static_cast<long long>(p.place_per) * p.k, all = static_cast<long long>(p.T) * p.k;
    const long long from = blockIdx.x * per, to = min(all, from + per);
    const int mine = static_cast<int>(blockIdx.x) / p.place_width;
    constexpr int kAhead = 4;
    int expert[kAhead], slot[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
        const long long i = from + threadIdx.x + u * kRouteThreads;
        expert[u] = i < to ? p.experts[i] : -1;
        slot[u] = i < to ? p.slots[i] : -1;
    }
    // Threads by expert, and those left over by cluster as well.
    int width = 32;
    while (width < p.E && width < kRouteThreads) width *= 2;
    const int parts = kRouteThreads / width, part = threadIdx.x / width;
    for (int e = threadIdx.x % width; e < p.E; e += width) {
        int sum = 0, sum_before = 0;
#pragma unroll 16
        for (int c = part; c < clusters; c += parts) {
            const int n = p.counts[static_cast<long long>(c) * p.E + e];
            sum += n;
            if (c < mine) sum_before += n;
        }
        atomicAdd(total + e, sum);
        atomicAdd(before + e, sum_before);
    }
    __syncthreads();
    exclusive_sums(total, p.E, base, blockIdx.x == 0 ? p.offsets : nullptr, scratch);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (expert[u] >= 0) p.slots[from + threadIdx.x + u * kRouteThreads] = slot[u] + base[expert[u]] + before[expert[u]];
    for (long long i = from + threadIdx.x + kAhead * kRouteThreads; i < to; i += kRouteThreads) {
        const int e = p.experts[i];
        if (e >= 0) p.slots[i] += base[e] + before[e];
    }
}

// ------------------------------------------------------------------ gradient

// With s the scores, W the weights and d their gradient (of the chosen):
//   sigmoid:  dl = scale d s (1 - s);  renormalised: dl = W (d - sum d W / scale) (1 - s)
//   softmax:  dl_e = s_e (scale d_e - sum_j scale d_j s_j) for every expert;
//             renormalised, a softmax over the chosen: dl = W (d - sum d W / scale)
// A warp a token; a lane holds the NPL neighbours that it writes.  16384 x 256 bf16, 8
// chosen: 5.4 us (3.1 TB/s of stores and reads); for every expert 6.7 us (9.4 and 12.5 with the chosen ones' parts
// sent to their lanes by shuffles).
constexpr int kGradWarps = 8;

template <int NPL, typename T>
__global__ void __launch_bounds__(32 * kGradWarps) route_grad_kernel(const RouteGradParams p) {
    constexpr int kQuad = NPL >= 4 ? 4 : 1;
    __shared__ __align__(16) float rows[kGradWarps][32 * NPL];
    const int lane = threadIdx.x & 31, first = lane * NPL;
    const long long t = static_cast<long long>(blockIdx.x) * kGradWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    float* const mine = rows[threadIdx.x >> 5];
#pragma unroll
    for (int i = 0; i < NPL; i += kQuad) {
        if constexpr (kQuad == 4)
            *reinterpret_cast<float4*>(mine + first + i) = make_float4(0.f, 0.f, 0.f, 0.f);
        else
            mine[first + i] = 0.f;
    }
    __syncwarp();
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    int e = -1;
    float d = 0.f, x = -INFINITY;
    if (lane < p.k) {
        e = __ldg(p.experts + t * p.k + lane);
        if (e >= p.E) e = -1;
        if (e >= 0) {
            d = __ldg(p.dweights + t * p.k + lane);
            x = to_f32(row[e]);
            if (x == -INFINITY) e = -1;
        }
    }
    const bool any = __any_sync(kAll, e >= 0);
    float v[NPL], g = 0.f;  // v: of every expert; g: more, of the lane's choice
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = 0.f;
    if (any) {
        const float top = warp_max(x);
        float s = 0.f, rest = 1.f;  // rest: 1 - s, of a sigmoid
        if (e >= 0 && p.sigmoid) {
            const float low = x > 0.f ? 0.f : x, tail = expf(-fabsf(x));
            const float inv = fast_reciprocal(1.f + tail);
            s = expf(low - (p.renormalize ? fminf(top, 0.f) : 0.f)) * inv;
            rest = (x > 0.f ? tail : 1.f) * inv;
        } else if (e >= 0) {
            s = expf(x - top);
        }
        if (p.renormalize) {
            s *= fast_reciprocal(warp_sum(s));
            const float mean = warp_sum(d * s);
            if (e >= 0) g = p.scale * s * (d - mean) * rest;
        } else if (p.sigmoid) {
            if (e >= 0) g = p.scale * d * s * rest;
        } else {
            float l[NPL];
            load_row<NPL>(row, lane * NPL, p.E, p.vec, l);
            float most = -INFINITY;
#pragma unroll
            for (int i = 0; i < NPL; ++i) most = fmaxf(most, l[i]);
            most = warp_max(most);
            float sum = 0.f;
            uint32_t open = 0;  // (zeros to the others, also where the gradients are not finite)
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                open |= l[i] == -INFINITY ? 0u : 1u << i;
                l[i] = l[i] == -INFINITY ? 0.f : fast_exp(l[i] - most);
                sum += l[i];
            }
            const float inv = fast_reciprocal(warp_sum(sum));
            s = e >= 0 ? fast_exp(x - most) * inv : 0.f;
            const float less = -p.scale * inv * warp_sum(d * s);
#pragma unroll
            for (int i = 0; i < NPL; ++i) v[i] = open >> i & 1 ? l[i] * less : 0.f;
            if (e >= 0) g = p.scale * s * d;
        }
        // The chosen experts' parts, by way of a row in shared memory.
        if (e >= 0) atomicAdd(mine + e, g);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NPL; i += kQuad) {
            if constexpr (kQuad == 4) {
                const float4 x = *reinterpret_cast<const float4*>(mine + first + i);
                v[i] += x.x, v[i + 1] += x.y, v[i + 2] += x.z, v[i + 3] += x.w;
            } else {
                v[i] += mine[first + i];
            }
        }
    }
    T* out = static_cast<T*>(p.dlogits) + t * p.ldd + first;
    constexpr int kBytes = NPL * static_cast<int>(sizeof(T)), kWord = kBytes < 16 ? kBytes : 16;
    if (kWord >= 4 && p.vec_out && first + NPL <= p.E) {
        alignas(16) T y[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) y[i] = from_f32<T>(v[i]);
#pragma unroll
        for (int i = 0; i < kBytes; i += kWord) {
            char* to = reinterpret_cast<char*>(out) + i;
            const char* of = reinterpret_cast<const char*>(y) + i;
            if constexpr (kWord == 16)
                *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(of);
            else if constexpr (kWord == 8)
                *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(of);
            else if constexpr (kWord == 4)
                *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(of);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (first + i < p.E) out[i] = from_f32<T>(v[i]);
    }
}

// f(T(), integral_constant<NPL>) for the type and the smallest NPL that holds E.
template <typename F>
int by_type_and_width(int type, int E, F f) {
    auto width = [&](auto zero) {
        if (E <= 32) return f(zero, std::integral_constant<int, 1>());
        if (E <= 64) return f(zero, std::integral_constant<int, 2>());
        if (E <= 128) return f(zero, std::integral_constant<int, 4>());
        if (E <= 256) return f(zero, std::integral_constant<int, 8>());
        if (E <= 512) return f(zero, std::integral_constant<int, 16>());
        return f(zero, std::integral_constant<int, 32>());
    };
    if (type == SGEMM_TYPE_F32) return width(0.f);
    if (type == SGEMM_TYPE_BF16) return width(__nv_bfloat16());
    return width(__half());
}

int launched() {
    if (cudaGetLastError() == cudaSuccess) return SGEMM_OK;
    return SGEMM_ERR_CUDA;
}

}  // namespace

RoutePlan route_plan(const RouteParams& p, int sms) {
    const int T = p.T;
    // Four lanes a token where they can, but for many experts and a token a warp at most: its 32 lanes are done sooner. us
    // (four lanes / a warp), 64 experts: 1 to 16 tokens 3.3 / 3.7, 64 4.1 / 4.6, 256 4.2 / 6.1, 512 6.5 / 9.5; 256 experts in
    // groups: 16 7.4 / 6.1, 64 8.9 / 6.2, 200 9.5 / 9.8, 512 12 / 16, 16384 28 / 40.
    const bool quads = p.k <= 8 && p.E <= 256 && (p.groups == 1 || (p.group_size >= 8 && !(p.group_size & (p.group_size - 1)))) &&
                       (p.E <= 64 || T > kRouteCluster * kRouteWarps);
    // One CTA or one cluster finishes by itself, which saves a launch.
    const int whole = quads ? kQuadStep : 2 * kRouteWarps;
    if (T <= kRouteWarps) return {1, 1, T, quads ? whole : kRouteWarps, quads};
    if (T <= (quads ? 1 : 2) * kRouteCluster * whole) {
        const int per = (T + kRouteCluster - 1) / kRouteCluster;
        return {1, kRouteCluster, per, !quads && per <= kRouteWarps ? kRouteWarps : whole, quads};
    }
    // Two CTAs an SM at once (four of a quarter of the threads), whole steps each.
    const int most = std::max(1, (quads ? 4 : 2) * sms / kRouteCluster) * kRouteCluster;
    const int per = ((T + most - 1) / most + whole - 1) / whole * whole;
    const int ctas = (T + per - 1) / per;
    return {(ctas + kRouteCluster - 1) / kRouteCluster, kRouteCluster, per, whole, quads};
}

int route(const RouteParams& given, const RoutePlan& plan, int type, cudaStream_t s) {
    RouteParams p = given;
    p.width = plan.width, p.per = plan.per, p.step = plan.step, p.steps = (plan.per + plan.step - 1) / plan.step;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(plan.clusters * plan.width));
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(plan.width);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = plan.width > 1 ? 1 : 0;
    const auto start = [&](auto kernel) {
        if (cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess) return static_cast<int>(SGEMM_OK);
        (void)cudaGetLastError();
        return static_cast<int>(SGEMM_ERR_CUDA);
    };
    // (the bias to the last lane's end: E up to a power of two from 32 on)
    const size_t smem = (5 * static_cast<size_t>(std::max(p.E, 32)) + kRouteWarps) * sizeof(int);
    const int rc = by_type_and_width(type, p.E, [&](auto zero, auto npl) {
        constexpr int NPL = decltype(npl)::value;
        using T = decltype(zero);
        if constexpr (NPL <= 8) {
            if (plan.quads) {
                constexpr int N = std::max(16, 8 * NPL);
                cfg.blockDim = dim3(kQuadThreads);
                cfg.dynamicSmemBytes = (4 * (N + 4) + 3 * static_cast<size_t>(p.E) + kQuadWarps) * sizeof(int);
                return start(route_quads_kernel<N, T>);
            }
        }
        const int lanes = p.group_size / NPL;
        p.group_lanes = 0;
        while (1 << p.group_lanes < lanes) ++p.group_lanes;
        if (p.groups > 1 && (p.group_size % NPL || 1 << p.group_lanes != lanes)) p.group_lanes = -1;
        cfg.blockDim = dim3(kRouteThreads);
        cfg.dynamicSmemBytes = smem;
        return start(route_kernel<NPL, T>);
    });
    if (rc != SGEMM_OK || !p.counts) return rc;
    // Places by CTA, or, of the smaller CTAs, by cluster.
    p.place_per = plan.quads ? plan.per * plan.width : plan.per;
    p.place_width = plan.quads ? 1 : plan.width;
    cfg.gridDim = dim3(static_cast<unsigned>(plan.clusters * p.place_width));
    cfg.blockDim = dim3(kRouteThreads);
    cfg.dynamicSmemBytes = smem;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, place_kernel, p, plan.clusters) != cudaSuccess) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

int route_grad(const RouteGradParams& p, int type, cudaStream_t s) {
    const unsigned ctas = static_cast<unsigned>((p.T + kGradWarps - 1) / kGradWarps);
    return by_type_and_width(type, p.E, [&](auto zero, auto npl) {
        route_grad_kernel<decltype(npl)::value, decltype(zero)><<<ctas, 32 * kGradWarps, 0, s>>>(p);
        return launched();
    });
}

}  // namespace gb300
