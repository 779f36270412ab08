// Internal interface of routing and of the rows' way to their experts
// (include/sgemm_routing.h): kernel parameters and launch functions.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace gb300 {

struct RouteParams {
    const void* logits;
    long long ld;
    const float* bias;  // null: none
    int T, E, k;
    int sigmoid, renormalize;
    int groups, top_groups, group_best;
    int group_size, group_lanes;  // E / groups; the lanes of a group's keys as a power of two, or -1 (set by route)
    float scale;
    int* experts;
    float* weights;
    int* offsets;
    int* slots;
    int vec;      // the rows begin on 16 bytes: whole vectors are loaded
    int width, per;    // CTAs of a cluster, tokens of a CTA (these to place_width are set by route)
    int steps, step;   // a CTA's steps, and the tokens of one
    int place_per, place_width;  // of the second kernel: tokens of a CTA, CTAs for a cluster's
    int* counts;      // clusters x E: choices of each expert (null: one cluster does it all)
};

// Warps of a CTA, and CTAs of a cluster where there is more than one.
constexpr int kRouteWarps = 16, kRouteCluster = 8;
constexpr int kQuadStep = 32;  // tokens of a CTA's step with four lanes a token

// The grid of a routing: clusters of `width` CTAs, each CTA's tokens, and those of a step; four lanes a token or a warp.
struct RoutePlan {
    int clusters, width, per, step;
    bool quads;
};
RoutePlan route_plan(const RouteParams& p, int sms);
int route(const RouteParams& p, const RoutePlan& plan, int type, cudaStream_t s);

struct RouteGradParams {
    const void* logits;
    long long ld;
    const int* experts;
    const float* dweights;
    void* dlogits;
    long long ldd;
    int T, E, k;
    int sigmoid, renormalize;
    float scale;
    int vec, vec_out;
};
int route_grad(const RouteGradParams& p, int type, cudaStream_t s);

// Rows to their slots and back (rows.cu).
struct RowsParams {
    const void* X;  // spread: X; gradient of a combination: dout
    long long ldx;
    const void* Y;  // combination and its gradient: rows by slot
    long long ldy;
    void* out;  // spread: Y; combination: out; its gradient: dY (may be null)
    long long ldo;
    const int* slots;
    const float* weights;  // null: ones
    float* dweights;       // may be null
    const int* used;       // &offsets[E]: rows of `out` from here on are zeroed (null: no `out`, or a combination's)
    int zero;              // this launch zeroes them (set by the launch functions)
    int T, k, R, H;
    int vec;  // elements a vector, as the operands' alignment allows
};
int rows_spread(const RowsParams& p, int type, int sms, cudaStream_t s);
int rows_combine(const RowsParams& p, int type, int sms, cudaStream_t s);
int rows_combine_grad(const RowsParams& p, int type, int sms, cudaStream_t s);

}  // namespace gb300
