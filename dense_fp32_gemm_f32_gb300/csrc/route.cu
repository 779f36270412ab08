// Routing of tokens to experts, and its gradient (include/sgemm_routing.h).
//
// A warp takes a token.  Lane l holds the scores of experts l * NPL .. l * NPL
// + NPL - 1, so that a row comes in with wide loads, a lane's experts are
// neighbours (groups span whole lanes) and the lowest of equal experts is the
// lowest lane's.  Scores are compared as unsigned keys in their order, 0 for
// an expert out of service: the warp's largest is then one redux instruction,
// and k of them with the lane's own largest kept up to date make the choice.
//
// What the choice is by.  Without a bias (and with group_best = 1) both scores
// grow with the logit, so logits are compared, exactly.  Otherwise float32
// scores decide where they are further apart than their errors; a token where
// two of those that decide are not goes through the same code in 64 bits
// (choose_again), so that no rounding of exp or of a sum moves a choice.
//
// Places.  A CTA takes tokens 32 at a time and sets a bit a token in a word of
// each chosen expert (an OR: its order does not matter); a choice's place
// among the expert's rows in this CTA is then the number of bits below its own
// plus those of the steps before.  The CTAs of a cluster add up their counts
// through distributed shared memory.  Up to 512 tokens are one cluster, which
// then knows all; else the clusters' counts go to a table, and place_kernel adds
// up, in a CTA a cluster, those of the clusters and of the experts before.
#include <algorithm>
#include <type_traits>

#include "../../include/sgemm_routing.h"
#include "experts_groups.cuh"
#include "ptx.cuh"
#include "routing.h"

namespace gb300 {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRouteWarps = 16, kRouteThreads = 32 * kRouteWarps;
constexpr int kRouteTokens = kRouteStep / kRouteWarps;  // tokens of a warp in a step

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

// Lane l's values of a row of E: elements l * NPL ..., -inf past the row's end.
template <int NPL, typename T>
__device__ __forceinline__ void load_row(const T* row, int E, bool vec, float (&v)[NPL]) {
    const int first = (threadIdx.x & 31) * NPL;
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

// The lane's keys, the largest first (equal ones by their number), and their
// numbers, 4 bits each.  Neighbours trade places, so that equal ones keep theirs.
template <int NPL, typename Key>
__device__ __forceinline__ uint32_t sort_lane(Key (&key)[NPL]) {
    static_assert(NPL <= 8, "4 bits each");
    uint32_t at[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) at[i] = i;
#pragma unroll
    for (int round = 0; round < NPL; ++round)
#pragma unroll
        for (int i = round & 1; i + 1 < NPL; i += 2) {
            const bool swap = key[i] < key[i + 1];
            const Key a = key[i], b = key[i + 1];
            key[i] = swap ? b : a;
            key[i + 1] = swap ? a : b;
            const uint32_t x = at[i], y = at[i + 1];
            at[i] = swap ? y : x;
            at[i + 1] = swap ? x : y;
        }
    uint32_t packed = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) packed |= at[i] << (4 * i);
    return packed;
}

// The two largest of four keys, (a >= b) and (c >= d), to a and b.
template <typename Key>
__device__ __forceinline__ void merge_two(Key& a, Key& b, Key c, Key d) {
    const Key low = min(a, c);
    a = max(a, c);
    b = max(low, max(b, d));
}

// The groups to choose from, a bit each: from the two best keys a, b of group g in
// lane g (0: none).  `sure`: whether that is certain; see choose().
template <typename V>
__device__ __forceinline__ unsigned choose_groups(const RouteParams& p, typename Keys<V>::Key a, typename Keys<V>::Key b,
                                                  bool checked, V near, bool& sure) {
    using K = Keys<V>;
    using Key = typename K::Key;
    Key score = 0;
    if ((threadIdx.x & 31) < p.groups && a) {
        V value = K::value(a);
        if (p.group_best == 2 && b) value += K::value(b);
        score = K::of(value);
    }
    unsigned kept = 0;
    Key last = 0;
    for (int i = 0; i < p.top_groups; ++i) {
        const Key best = K::most(score);
        if (best == 0) return kept;
        const unsigned lane = __ffs(__ballot_sync(kAll, score == best)) - 1;
        kept |= 1u << lane;
        if ((threadIdx.x & 31) == lane) score = 0;
        last = best;
    }
    if (checked) {  // (what is among them or not is decided at their end alone)
        const Key next = K::most(score);
        if (next && !(K::value(last) - K::value(next) > 2 * near)) sure = false;
    }
    return kept;
}

// Of a token's keys (0: out of service), the k best in order: lane j's result
// is the j-th expert, -1 where there is none.  checked: `sure` is false if two
// values that decide lie within `near` of one another (the result is then not
// to be used).
template <int NPL, typename V>
__device__ __forceinline__ int choose(typename Keys<V>::Key (&key)[NPL], const RouteParams& p, bool checked, V near,
                                      bool& sure) {
    using K = Keys<V>;
    using Key = typename K::Key;
    constexpr bool SORTED = NPL <= 8 && sizeof(V) == 4;
    const int lane = threadIdx.x & 31, first = lane * NPL;
    const int size = p.groups > 1 ? p.E / p.groups : 0, lanes = size / NPL;
    const bool whole = size % NPL == 0 && (lanes & (lanes - 1)) == 0;  // a power of two of whole lanes a group
    sure = true;
    if (p.groups > 1 && !(SORTED && whole)) {
        Key a = 0, b = 0;
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
        const unsigned kept = choose_groups<V>(p, a, b, checked, near, sure);
        int g = first / size, rest = first - g * size;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            if (g >= p.groups || !(kept >> g & 1)) key[i] = 0;
            if (++rest == size) rest = 0, ++g;
        }
    }
    uint32_t at = 0;  // sorted: numbers of the lane's keys, the first in the low bits; else the largest one's
    Key m = 0;
    auto lead = [&] {
        m = key[0], at = 0;
#pragma unroll
        for (int i = 1; i < NPL; ++i)
            if (key[i] > m) m = key[i], at = i;
    };
    if constexpr (SORTED) {
        at = sort_lane(key);
        m = key[0];
        if (p.groups > 1 && whole) {
            Key a = m, b = NPL > 1 ? key[NPL > 1 ? 1 : 0] : Key{0};
            for (int d = 1; d < lanes; d *= 2) merge_two(a, b, __shfl_xor_sync(kAll, a, d), __shfl_xor_sync(kAll, b, d));
            const int from = (lane * lanes) & 31;
            a = __shfl_sync(kAll, a, from);
            b = __shfl_sync(kAll, b, from);
            const unsigned kept = choose_groups<V>(p, a, b, checked, near, sure);
            const int g = lane / lanes;
            if (!(kept >> g & 1)) m = 0;  // (lanes past the last group hold no keys)
        }
    } else {
        lead();
    }
    if (!sure) return -1;
    Key before = 0;
    int mine = -1;
    for (int j = 0; j < p.k + (checked ? 1 : 0); ++j) {
        const Key best = K::most(m);
        if (best == 0) break;
        if (checked && j > 0 && !(K::value(before) - K::value(best) > near)) {
            sure = false;
            return -1;
        }
        if (j == p.k) break;
        before = best;
        const int from = __ffs(__ballot_sync(kAll, m == best)) - 1;
        const int e = __shfl_sync(kAll, first + static_cast<int>(SORTED ? at & 15 : at), from);
        if (lane == j) mine = e;
        if (lane == from) {
            if constexpr (SORTED) {
#pragma unroll
                for (int i = 0; i + 1 < NPL; ++i) key[i] = key[i + 1];
                key[NPL - 1] = 0;
                at >>= 4;
                m = key[0];
            } else {
#pragma unroll
                for (int i = 0; i < NPL; ++i)
                    if (i == static_cast<int>(at)) key[i] = 0;
                lead();
            }
        }
    }
    return mine;
}

// The choice in 64 bits.
template <int NPL, typename T>
__device__ __noinline__ int choose_again(const RouteParams& p, const T* row) {
    float l[NPL];
    load_row<NPL>(row, p.E, p.vec, l);
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) top = fmaxf(top, l[i]);
    top = warp_max(top);
    double sum = 0;
    if (!p.sigmoid) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) sum += l[i] == -INFINITY ? 0. : exp(static_cast<double>(l[i]) - top);
        sum = warp_sum(sum);
    }
    const int first = (threadIdx.x & 31) * NPL;
    unsigned long long key[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        key[i] = 0;
        if (l[i] != -INFINITY) {
            const double x = l[i];
            double c = p.sigmoid ? 1. / (1. + exp(-x)) : exp(x - top) / sum;
            if (p.bias) c += __ldg(p.bias + first + i);
            if (c != -INFINITY) key[i] = Keys<double>::of(c);
        }
    }
    bool sure;
    return choose<NPL, double>(key, p, false, 0., sure);
}

// A token's experts and weights, the j-th in lane j, from its row (l: the lane's part).
template <int NPL, typename T>
__device__ __forceinline__ int route_token(const RouteParams& p, const T* row, const float (&l)[NPL],
                                           const float (&bias)[NPL], float& weight) {
    const bool by_logit = !p.bias && (p.groups == 1 || p.group_best == 1);
    float top = 0.f, sum = 0.f;
    uint32_t key[NPL];
    if (!p.sigmoid && (!by_logit || !p.renormalize)) {
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i) top = fmaxf(top, l[i]);
        top = warp_max(top);
#pragma unroll
        for (int i = 0; i < NPL; ++i) sum += l[i] == -INFINITY ? 0.f : expf(l[i] - top);
        sum = warp_sum(sum);
    }
    bool sure;
    int e;
    if (by_logit) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) key[i] = l[i] == -INFINITY ? 0u : Keys<float>::of(l[i]);
        e = choose<NPL, float>(key, p, false, 0.f, sure);
    } else {
        // Errors.  Softmax: exp(l - top) is off by |l - top| 2^-24 (the
        // difference's rounding) and 2 units; times exp(l - top), the former is
        // largest at |l - top| = 1; the sum by 12 units and by the mean of
        // |l - top| over the softmax, below log 1024 = 7: in all below 2^-19 of
        // the largest score.  Sigmoid: below 2^-21.  Then half a unit of the
        // sum with the bias.  Two values are in order when they are further
        // apart than both errors.
        const float inv = 1.f / sum;
        float size = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            key[i] = 0;
            if (l[i] != -INFINITY) {
                const float s = p.sigmoid ? __fdividef(1.f, 1.f + expf(-l[i])) : expf(l[i] - top) * inv;
                const float c = s + bias[i];
                size = fmaxf(size, fabsf(c));
                if (c != -INFINITY) key[i] = Keys<float>::of(c);
            }
        }
        size = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(size)));
        const float near = 0x1p-22f * size + (p.sigmoid ? 0x1p-20f : 0x1p-18f * inv);
        e = choose<NPL, float>(key, p, true, near, sure);
        if (!sure) e = choose_again<NPL>(p, row);
    }
    // Weights.  sigmoid(l) = e^min(l, 0) / (1 + e^-|l|): with the largest chosen
    // logit's e^min(l, 0) taken out, the renormalised ones are ratios of
    // numbers near 1 however small the scores are.
    const float x = e >= 0 ? to_f32(row[e]) : -INFINITY;
    float s = 0.f;
    const float lead = p.renormalize ? warp_max(x) : top;
    if (e >= 0) {
        if (p.sigmoid) {
            const float low = x > 0.f ? 0.f : x;
            s = expf(low - (p.renormalize ? fminf(lead, 0.f) : 0.f)) / (1.f + expf(-fabsf(x)));
        } else {
            s = expf(x - lead);
            if (sum != sum) s = sum;  // (a NaN or +inf that was not chosen)
        }
    }
    if (p.renormalize) sum = warp_sum(s);
    weight = e < 0 ? 0.f : p.sigmoid && !p.renormalize ? p.scale * s : p.scale * s / sum;
    return e;
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

// CLUSTER: CTAs of a cluster (their count of each expert's choices is summed
// through distributed shared memory).  With p.counts there are several clusters,
// which leave their sums there for place_kernel; else the one finishes the places.
template <int NPL, typename T, int CLUSTER>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p) {
    extern __shared__ int shared[];
    int* const mask = shared;             // E: this step's tokens
    int* const count = shared + p.E;      // E: choices of the steps before
    int* const before = shared + 2 * p.E; // E: of the cluster's CTAs before this one, then all that come before
    int* const scratch = shared + 3 * p.E;  // a word a warp
    grid_dependency_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) mask[e] = count[e] = 0;
    float bias[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane * NPL + i;
        bias[i] = p.bias && e < p.E ? __ldg(p.bias + e) : 0.f;
    }
    __syncthreads();
    const long long begin = static_cast<long long>(blockIdx.x) * p.steps * kRouteStep;
    int mine[kRouteTokens] = {}, rank[kRouteTokens] = {};  // of the last step
    for (int step = 0; step < p.steps; ++step) {
        const long long t0 = begin + step * kRouteStep + warp;
        auto row = [&](int i) { return static_cast<const T*>(p.logits) + (t0 + i * kRouteWarps) * p.ld; };
        float l[NPL], next[NPL];
        if (t0 < p.T) load_row<NPL>(row(0), p.E, p.vec, l);
#pragma unroll
        for (int i = 0; i < kRouteTokens; ++i) {
            const long long t = t0 + i * kRouteWarps;
            const bool more = i + 1 < kRouteTokens && t + kRouteWarps < p.T;
            if (NPL <= 8 && more) load_row<NPL>(row(i + 1), p.E, p.vec, next);  // (beside this token's work)
            int e = -1;
            if (t < p.T) {
                float w;
                e = route_token<NPL, T>(p, row(i), l, bias, w);
                if (lane < p.k) {
                    p.experts[t * p.k + lane] = e;
                    p.weights[t * p.k + lane] = w;
                    if (e >= 0) atomicOr(mask + e, 1 << (warp + i * kRouteWarps));
                }
            }
            mine[i] = lane < p.k ? e : -1;
            if (NPL > 8 && more) load_row<NPL>(row(i + 1), p.E, p.vec, next);
            if (more) {
#pragma unroll
                for (int j = 0; j < NPL; ++j) l[j] = next[j];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRouteTokens; ++i) {
            const long long t = t0 + i * kRouteWarps;
            const unsigned below = (1u << (warp + i * kRouteWarps)) - 1;
            rank[i] = mine[i] < 0 ? -1 : count[mine[i]] + __popc(mask[mine[i]] & below);
            if (step + 1 < p.steps && t < p.T && lane < p.k) p.slots[t * p.k + lane] = rank[i];
        }
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
            count[e] += __popc(mask[e]);
            mask[e] = 0;
        }
        __syncthreads();
    }
    // What comes before this CTA's choices of an expert, in the cluster.
    int* total = count;
    if constexpr (CLUSTER > 1) {
        const int of = static_cast<int>(cluster_ctarank());
        cluster_sync_all();
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
            const uint32_t at = smem_addr(count + e);
            int sum = 0, mine_from = 0;
#pragma unroll
            for (int q = 0; q < CLUSTER; ++q) {
                if (q == of) mine_from = sum;
                sum += ld_shared_cluster_s32(map_shared_rank(at, q));
            }
            before[e] = mine_from;
            mask[e] = sum;
            if (p.counts && of == 0) p.counts[static_cast<long long>(blockIdx.x / CLUSTER) * p.E + e] = sum;
        }
        total = mask;
        cluster_sync_all();  // (nobody reads this CTA's counts after this)
    } else {
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads) before[e] = 0;
        __syncthreads();
    }
    if (!p.counts) {
        int* const base = CLUSTER > 1 ? count : mask;
        exclusive_sums(total, p.E, base, blockIdx.x == 0 ? p.offsets : nullptr, scratch);
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads) before[e] += base[e];
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kRouteTokens; ++i) {
        const long long t = begin + (p.steps - 1) * kRouteStep + warp + i * kRouteWarps;
        if (t < p.T && lane < p.k) p.slots[t * p.k + lane] = mine[i] < 0 ? -1 : rank[i] + before[mine[i]];
    }
    if (p.steps > 1) {  // the steps before the last, whose places are in memory
        const long long from = begin * p.k, to = min(static_cast<long long>(p.T), begin + (p.steps - 1) * kRouteStep) * p.k;
        for (long long i = from + threadIdx.x; i < to; i += kRouteThreads) {
            const int e = p.experts[i];
            if (e >= 0) p.slots[i] += before[e];
        }
    }
}

// Places within a cluster's rows of an expert to places among all rows; a CTA a cluster.
__global__ void __launch_bounds__(kRouteThreads) place_kernel(const RouteParams p, int clusters) {
    extern __shared__ int shared[];
    int* const total = shared;
    int* const before = shared + p.E;
    int* const base = shared + 2 * p.E;
    int* const scratch = shared + 3 * p.E;
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) total[e] = before[e] = 0;
    __syncthreads();
    grid_dependency_wait();
    // Threads by expert, and those left over by CTA as well.
    int width = 32;
    while (width < p.E && width < kRouteThreads) width *= 2;
    const int parts = kRouteThreads / width, part = threadIdx.x / width;
    for (int e = threadIdx.x % width; e < p.E; e += width) {
        int all = 0, mine = 0;
#pragma unroll 8
        for (int c = part; c < clusters; c += parts) {
            const int n = p.counts[static_cast<long long>(c) * p.E + e];
            all += n;
            if (c < static_cast<int>(blockIdx.x)) mine += n;
        }
        atomicAdd(total + e, all);
        atomicAdd(before + e, mine);
    }
    __syncthreads();
    exclusive_sums(total, p.E, base, blockIdx.x == 0 ? p.offsets : nullptr, scratch);
    const long long per = static_cast<long long>(p.steps) * kRouteStep * kRouteCluster * p.k, all = static_cast<long long>(p.T) * p.k;
    const long long from = blockIdx.x * per, to = min(all, from + per);
    for (long long i = from + threadIdx.x; i < to; i += kRouteThreads) {
        const int e = p.experts[i];
        if (e >= 0) p.slots[i] += base[e] + before[e];
    }
}

// ------------------------------------------------------------------ gradient

// With s the scores, W the weights and d their gradient (of the chosen):
//   sigmoid:  dl = scale d s (1 - s);  renormalised: dl = W (d - sum d W / scale) (1 - s)
//   softmax:  dl_e = s_e (scale d_e - sum_j scale d_j s_j) for every expert;
//             renormalised, a softmax over the chosen: dl = W (d - sum d W / scale)
// A warp a token; a lane holds the NPL neighbours that it writes.
constexpr int kGradWarps = 8;

template <int NPL, typename T>
__global__ void __launch_bounds__(32 * kGradWarps) route_grad_kernel(const RouteGradParams p) {
    const int lane = threadIdx.x & 31, first = lane * NPL;
    const long long t = static_cast<long long>(blockIdx.x) * kGradWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
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
            s = expf(low - (p.renormalize ? fminf(top, 0.f) : 0.f)) / (1.f + tail);
            rest = (x > 0.f ? tail : 1.f) / (1.f + tail);
        } else if (e >= 0) {
            s = expf(x - top);
        }
        if (p.renormalize) {
            s /= warp_sum(s);
            const float mean = warp_sum(d * s);
            if (e >= 0) g = p.scale * s * (d - mean) * rest;
        } else if (p.sigmoid) {
            if (e >= 0) g = p.scale * d * s * rest;
        } else {
            float l[NPL];
            load_row<NPL>(row, p.E, p.vec, l);
            float most = -INFINITY;
#pragma unroll
            for (int i = 0; i < NPL; ++i) most = fmaxf(most, l[i]);
            most = warp_max(most);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                l[i] = l[i] == -INFINITY ? 0.f : expf(l[i] - most);
                sum += l[i];
            }
            sum = warp_sum(sum);
            s = e >= 0 ? expf(x - most) / sum : 0.f;
            const float mean = warp_sum(d * s);
#pragma unroll
            for (int i = 0; i < NPL; ++i) v[i] = -p.scale * (l[i] / sum) * mean;
            if (e >= 0) g = p.scale * s * d;
        }
        for (int j = 0; j < p.k; ++j) {
            const int at = __shfl_sync(kAll, e, j);
            const float more = __shfl_sync(kAll, g, j);
            const int i0 = at - first;
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (at >= 0 && i == i0) v[i] += more;
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

RoutePlan route_plan(int T, int sms) {
    const int steps = (T + kRouteStep - 1) / kRouteStep;
    if (steps == 1) return {1, 1, 1};
    // One cluster finishes by itself, which saves a launch: up to two steps of it.
    const int least = (steps + kRouteCluster - 1) / kRouteCluster;
    if (least <= 2) return {1, kRouteCluster, least};
    // About three CTAs an SM at once.
    const int most = std::max(1, 3 * sms / kRouteCluster);
    const int each = (least + most - 1) / most;
    return {(least + each - 1) / each, kRouteCluster, each};
}

int route(const RouteParams& p, const RoutePlan& plan, int type, cudaStream_t s) {
    const size_t smem = (3 * static_cast<size_t>(p.E) + kRouteWarps) * sizeof(int);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(plan.clusters * plan.width));
    cfg.blockDim = dim3(kRouteThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(plan.width);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = plan.width > 1 ? 1 : 0;
    const int rc = by_type_and_width(type, p.E, [&](auto zero, auto npl) {
        constexpr int NPL = decltype(npl)::value;
        using T = decltype(zero);
        const auto kernel = plan.width > 1 ? route_kernel<NPL, T, kRouteCluster> : route_kernel<NPL, T, 1>;
        if (cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess) return static_cast<int>(SGEMM_OK);
        (void)cudaGetLastError();
        return static_cast<int>(SGEMM_ERR_CUDA);
    });
    if (rc != SGEMM_OK || !p.counts) return rc;
    cfg.gridDim = dim3(static_cast<unsigned>(plan.clusters));
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
