// The entry points of include/sgemm_routing.h: argument checks and launches.
#include "../../include/sgemm_routing.h"
#include "api_internal.h"
#include "experts.h"
#include "routing.h"
#include "views.h"

using namespace gb300;
using namespace gb300::detail;

namespace {

View ints_view(const void* p, int64_t n) { return {p, 1, 1, n, n, 0, 4}; }

// No output overlaps an input or another output.
template <size_t I, size_t O>
bool apart(const View (&in)[I], const View (&out)[O]) {
    for (size_t i = 0; i < O; ++i) {
        for (const View& v : in)
            if (overlap(out[i], v)) return false;
        for (size_t j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return false;
    }
    return true;
}

// Whether each row of `v` begins on 16 bytes.
bool whole_vectors(const View& v) { return row_alignment(v.p, v.size, v.rows > 1 ? v.ld : 0, 0) == 16; }

bool route_sizes_ok(int type, int score, int T, int E, int k) {
    return type_ok(type) && (score == SGEMM_SCORE_SOFTMAX || score == SGEMM_SCORE_SIGMOID) && T >= 0 && T <= kMost &&
           E >= 1 && E <= SGEMM_ROUTE_MAX_EXPERTS && k >= 1 && k <= SGEMM_ROUTE_MAX_CHOICES && k <= E &&
           static_cast<int64_t>(T) * k <= kMost;
}

// The largest vector, in elements, that the rows of all of `v` allow (those of a
// single row as well: every row's first element is what counts).
int vector_of(std::initializer_list<View> v) {
    int bytes = 16, size = 4;
    for (const View& x : v)
        if (x.p && !x.empty()) {
            bytes = std::min(bytes, row_alignment(x.p, x.size, x.rows > 1 ? x.ld : 0, 0));
            size = x.size;
        }
    return std::max(1, bytes / size);
}

bool rows_sizes_ok(int type, int T, int k, int R, int H) {
    return type_ok(type) && T >= 0 && k >= 0 && R >= 0 && H >= 0 && T <= kMost && k <= kMost && R <= kMost &&
           H <= kMost && static_cast<int64_t>(T) * k <= kMost;
}

}  // namespace

extern "C" {

int sgemm_route(int type, int score, int T, int E, int k, const void* logits, int64_t ld, const float* bias, int groups,
                int top_groups, int group_best, int renormalize, float scale, int* experts, float* weights,
                int* offsets, int* slots, void* stream) {
    if (!route_sizes_ok(type, score, T, E, k)) return SGEMM_ERR_INVALID_ARG;
    if (groups < 1 || groups > SGEMM_ROUTE_MAX_GROUPS || E % groups || top_groups < 1 || top_groups > groups ||
        (group_best != 1 && group_best != 2) || (renormalize != 0 && renormalize != 1))
        return SGEMM_ERR_INVALID_ARG;
    const View in[] = {{logits, 1, T, E, ld, 0, type_bytes(type)}, ints_view(bias, bias ? E : 0)};
    const int64_t n = static_cast<int64_t>(T) * k;
    const View out[] = {ints_view(experts, n), ints_view(weights, n), ints_view(slots, n), ints_view(offsets, E + 1)};
    if (!in[0].ok(in[0].size) || !in[1].ok(4)) return SGEMM_ERR_INVALID_ARG;
    for (const View& v : out)
        if (!v.ok(4)) return SGEMM_ERR_INVALID_ARG;
    if (!apart(in, out)) return SGEMM_ERR_INVALID_ARG;
    int dev = 0;
    DeviceState* st = nullptr;
    int rc = current_device(&dev, &st);
    if (rc != SGEMM_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) return zero_rows(offsets, 1, 1, E + 1, E + 1, 0, 4, s);
    RouteParams p = {};
    p.logits = logits, p.ld = ld, p.bias = bias;
    p.T = T, p.E = E, p.k = k;
    p.sigmoid = score == SGEMM_SCORE_SIGMOID, p.renormalize = renormalize, p.scale = scale;
    p.groups = top_groups < groups ? groups : 1;  // (all groups: no choice among them)
    p.top_groups = top_groups, p.group_best = group_best, p.group_size = E / groups;
    p.experts = experts, p.weights = weights, p.offsets = offsets, p.slots = slots;
    p.vec = whole_vectors(in[0]);
    const RoutePlan plan = route_plan(p, st->sm_count);
    if (plan.clusters > 1) {
        cudaMemPool_t pool = workspace_pool(dev, *st);
        void* ws = nullptr;
        if (!pool || cudaMallocFromPoolAsync(&ws, sizeof(int) * plan.clusters * E, pool, s) != cudaSuccess) {
            (void)cudaGetLastError();
            return SGEMM_ERR_CUDA;
        }
        p.counts = static_cast<int*>(ws);
    }
    rc = route(p, plan, type, s);
    if (p.counts) (void)cudaFreeAsync(p.counts, s);
    return rc;
}

int sgemm_route_grad(int type, int score, int T, int E, int k, const void* logits, int64_t ld, const int* experts,
                     const float* dweights, int renormalize, float scale, void* dlogits, int64_t ldd, void* stream) {
    if (!route_sizes_ok(type, score, T, E, k) || (renormalize != 0 && renormalize != 1)) return SGEMM_ERR_INVALID_ARG;
    const int64_t n = static_cast<int64_t>(T) * k;
    const View in[] = {{logits, 1, T, E, ld, 0, type_bytes(type)}, ints_view(experts, n), ints_view(dweights, n)};
    const View out[] = {{dlogits, 1, T, E, ldd, 0, type_bytes(type)}};
    if (!in[0].ok(in[0].size) || !in[1].ok(4) || !in[2].ok(4) || !out[0].ok(out[0].size) || !apart(in, out))
        return SGEMM_ERR_INVALID_ARG;
    if (T == 0) return SGEMM_OK;
    int dev = 0;
    DeviceState* st = nullptr;
    const int rc = current_device(&dev, &st);
    if (rc != SGEMM_OK) return rc;
    RouteGradParams p = {};
    p.logits = logits, p.ld = ld;
    p.experts = experts, p.dweights = dweights, p.dlogits = dlogits, p.ldd = ldd;
    p.T = T, p.E = E, p.k = k;
    p.sigmoid = score == SGEMM_SCORE_SIGMOID, p.renormalize = renormalize, p.scale = scale;
    p.vec = whole_vectors(in[0]), p.vec_out = whole_vectors(out[0]);
    return route_grad(p, type, static_cast<cudaStream_t>(stream));
}

int sgemm_spread(int type, int T, int k, int R, int H, const void* X, int64_t ldx, const int* slots, int E,
                 const int* offsets, void* Y, int64_t ldy, void* stream) {
    if (!rows_sizes_ok(type, T, k, R, H) || E < 0 || E > kMost || !offsets_ok(offsets)) return SGEMM_ERR_INVALID_ARG;
    const int size = type_bytes(type);
    const View in[] = {{X, 1, T, H, ldx, 0, size}, ints_view(slots, static_cast<int64_t>(T) * k), ints_view(offsets, E + 1)};
    const View out[] = {{Y, 1, R, H, ldy, 0, size}};
    if (!in[0].ok(size) || !in[1].ok(4) || !out[0].ok(size) || !apart(in, out)) return SGEMM_ERR_INVALID_ARG;
    if (out[0].empty()) return SGEMM_OK;
    int dev = 0;
    DeviceState* st = nullptr;
    const int rc = current_device(&dev, &st);
    if (rc != SGEMM_OK) return rc;
    RowsParams p = {};
    p.X = X, p.ldx = ldx, p.out = Y, p.ldo = ldy, p.slots = slots, p.used = offsets + E;
    p.T = T, p.k = k, p.R = R, p.H = H;
    p.vec = vector_of({in[0], out[0]});
    return rows_spread(p, type, st->sm_count, static_cast<cudaStream_t>(stream));
}

int sgemm_combine(int type, int T, int k, int R, int H, const void* Y, int64_t ldy, const int* slots,
                  const float* weights, void* out_, int64_t ldo, void* stream) {
    if (!rows_sizes_ok(type, T, k, R, H)) return SGEMM_ERR_INVALID_ARG;
    const int size = type_bytes(type);
    const int64_t n = static_cast<int64_t>(T) * k;
    const View in[] = {{Y, 1, R, H, ldy, 0, size}, ints_view(slots, n), ints_view(weights, weights ? n : 0)};
    const View out[] = {{out_, 1, T, H, ldo, 0, size}};
    if (!in[0].ok(size) || !in[1].ok(4) || !in[2].ok(4) || !out[0].ok(size) || !apart(in, out))
        return SGEMM_ERR_INVALID_ARG;
    if (out[0].empty()) return SGEMM_OK;
    int dev = 0;
    DeviceState* st = nullptr;
    const int rc = current_device(&dev, &st);
    if (rc != SGEMM_OK) return rc;
    RowsParams p = {};
    p.Y = Y, p.ldy = ldy, p.out = out_, p.ldo = ldo, p.slots = slots, p.weights = weights;
    p.T = T, p.k = k, p.R = R, p.H = H;
    p.vec = vector_of({in[0], out[0]});
    return rows_combine(p, type, st->sm_count, static_cast<cudaStream_t>(stream));
}

int sgemm_combine_grad(int type, int T, int k, int R, int H, const void* dout, int64_t ldd, const void* Y, int64_t ldy,
                       const int* slots, const float* weights, int E, const int* offsets, void* dY, int64_t lddy,
                       float* dweights, void* stream) {
    if (!rows_sizes_ok(type, T, k, R, H) || E < 0 || E > kMost) return SGEMM_ERR_INVALID_ARG;
    const int size = type_bytes(type);
    const int64_t n = static_cast<int64_t>(T) * k;
    if (dY && !offsets_ok(offsets)) return SGEMM_ERR_INVALID_ARG;
    const View in[] = {{dout, 1, T, H, ldd, 0, size}, {Y, 1, dweights ? R : 0, H, ldy, 0, size}, ints_view(slots, n),
                       ints_view(weights, weights ? n : 0), ints_view(offsets, dY ? E + 1 : 0)};
    const View out[] = {{dY, 1, dY ? R : 0, H, lddy, 0, size}, ints_view(dweights, dweights ? n : 0)};
    if (!in[0].ok(size) || !in[1].ok(size) || !in[2].ok(4) || !in[3].ok(4) || !out[0].ok(size) || !out[1].ok(4) ||
        !apart(in, out))
        return SGEMM_ERR_INVALID_ARG;
    if (out[0].empty() && out[1].empty()) return SGEMM_OK;
    int dev = 0;
    DeviceState* st = nullptr;
    const int rc = current_device(&dev, &st);
    if (rc != SGEMM_OK) return rc;
    RowsParams p = {};
    p.X = dout, p.ldx = ldd, p.Y = Y, p.ldy = ldy, p.slots = slots, p.weights = weights;
    p.out = out[0].empty() ? nullptr : dY, p.ldo = lddy, p.dweights = out[1].empty() ? nullptr : dweights;
    p.used = p.out ? offsets + E : nullptr;
    p.T = T, p.k = k, p.R = R, p.H = H;
    p.vec = vector_of({in[0], in[1], out[0]});
    return rows_combine_grad(p, type, st->sm_count, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
