// The entry point of include/sgemm_ortho.h: argument checks.
#include <cmath>

#include "../../include/sgemm_ortho.h"
#include "api_internal.h"
#include "ortho.h"
#include "views.h"

using namespace gb300;
using namespace gb300::detail;

namespace {

// The largest |b u + c u^2| and |a s + b s^3 + c s^5| for s in [0, most], u = s^2:
// at the ends, and where the derivatives are zero.
double largest_correction(double b, double c, double most, double a = 0) {  // (a: |a + b u + c u^2|)
    const double u = most * most;
    double top = std::fmax(std::fabs(a), std::fabs(a + b * u + c * u * u));
    if (c != 0) {
        const double at = -b / (2 * c);
        if (at > 0 && at < u) top = std::fmax(top, std::fabs(a + b * at + c * at * at));
    }
    return top;
}
double largest_value(double a, double b, double c, double most) {
    auto value = [&](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
    double top = value(most);
    auto root = [&](double u) {
        if (u > 0 && u < most * most) top = std::fmax(top, value(std::sqrt(u)));
    };
    if (c != 0) {  // 5 c u^2 + 3 b u + a = 0
        const double disc = 9 * b * b - 20 * a * c;
        if (disc >= 0) {
            root((-3 * b + std::sqrt(disc)) / (10 * c));
            root((-3 * b - std::sqrt(disc)) / (10 * c));
        }
    } else if (b != 0) {
        root(-a / (3 * b));
    }
    return top;
}

// Whether the polynomial keeps every singular value that can occur within 2, and
// what is added within 15 (see the scales in ortho_tc.cuh); `growth`: of |p(s) / s| as a power of two.
bool polynomial_ok(int steps, double a, double b, double c, int* growth) {
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
    double most = 1;
    for (int i = 0; i < steps; ++i) {
        if (!(largest_correction(b, c, most) <= 15)) return false;
        const double next = largest_value(a, b, c, most);
        if (!(next <= 2)) return false;
        most = std::fmax(most, next);
    }
    const double raises = largest_correction(b, c, most, a);  // (at most 32: of a, b + c and a + b + c two are bounded)
    for (*growth = 0; std::ldexp(1., *growth) < raises;) ++*growth;
    return true;
}

// A side's most.  The tensor cores cut a sum each time that they add to it, always towards zero, n / 16 times over a
// row of n where one plane is multiplied (two: at most 32 times): the bf16 result is then off by 1.7e-3 of its norm (1.7e-3 of it its rounding) up to 65536 columns, 2.1e-3 at
// 262144, 5.1e-3 at a million and 2.9e-2 at seven.
constexpr int kLongest = 1 << 18;

// The flag of products with one f16 value an operand out of `type`, where that may have it.
bool take_quick(int* type, int* parts) {
    const bool quick = (*type & SGEMM_ORTHO_QUICK) != 0;
    *type &= ~SGEMM_ORTHO_QUICK;
    if (quick) *parts = 1;
    return !quick || *type == SGEMM_TYPE_BF16;
}

bool sizes_ok(int type, int E, int M, int N, int steps) {
    if (!type_ok(type) || E < 0 || M < 0 || N < 0 || E > kOrthoMostMatrices || M > kLongest || N > kLongest || steps < 1 || steps > 64)
        return false;
    constexpr int64_t most = int64_t{1} << 46;  // elements
    return N == 0 || E == 0 || (M <= most / N && static_cast<int64_t>(M) * N <= most / E);
}

}  // namespace

extern "C" int64_t sgemm_orthogonalize_workspace(int type, int E, int M, int N, int steps) {
    int parts = 2;
    if (!take_quick(&type, &parts) || !sizes_ok(type, E, M, N, steps)) return -1;
    if (E == 0 || M == 0 || N == 0 || ortho_always_small(M, N)) return 0;
    return ortho_layout(E, M, N, steps, parts).bytes;
}

extern "C" int sgemm_orthogonalize(int type, int E, int M, int N, const void* G, int64_t ldg, int64_t stride_g, int steps,
                                   float a, float b, float c, double eps, void* out, int64_t ldo, int64_t stride_out,
                                   void* workspace, int64_t workspace_bytes, void* stream) {
    const int asked = type;
    int parts = 2, growth = 0;
    if (!take_quick(&type, &parts) || !sizes_ok(type, E, M, N, steps) || !(eps >= 0) || !std::isfinite(eps) || !polynomial_ok(steps, a, b, c, &growth))
        return SGEMM_ERR_INVALID_ARG;
    const int size = type_bytes(type);
    const View g{G, E, M, N, ldg, stride_g, size}, o{out, E, M, N, ldo, stride_out, size};
    if (!g.ok(size) || !o.ok(size) || overlap(g, o)) return SGEMM_ERR_INVALID_ARG;
    if (o.empty()) return SGEMM_OK;
    const int64_t needed = sgemm_orthogonalize_workspace(asked, E, M, N, steps);
    const View ws{workspace, 1, 1, needed, needed, 0, 1};
    if (workspace_bytes < needed || !ws.ok(256) || overlap(ws, g) || overlap(ws, o)) return SGEMM_ERR_INVALID_ARG;
    int dev = 0;
    DeviceState* st = nullptr;
    const int rc = experts_device(&dev, &st);
    if (rc != SGEMM_OK) return rc;
    const OrthoCall call = {G, ldg, stride_g, out, ldo, stride_out, type, E, M, N, steps, parts, a, b, c, growth, eps, workspace};
    return orthogonalize(call, *st, static_cast<cudaStream_t>(stream));
}
