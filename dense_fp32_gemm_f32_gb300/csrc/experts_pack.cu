// Copies of operands that the tensor maps cannot read: 16-bit rows off the
// 16-byte grid into pitched rows, and float32 operands into three bf16 parts,
//     x0 = bf16(x), x1 = bf16(x - x0), x2 = bf16(x - x0 - x1),
// each difference exact in float32 (x's 24 bits less the 8 leading ones of
// what is left, twice), so that what the parts miss is below 2^-25 |x|.  A
// finite x that bf16 would round to infinity is cut instead; the parts of a
// non-finite x are x, 0, 0.  Weights of experts without rows are not copied.
//
// Bound by bytes: 4 read and 6 written a float32, 2 and 2 a 16-bit value.  A
// thread takes 8 neighbouring elements of a row: whole 16-byte blocks of HBM
// (the block that a row begins in the middle of included: it lies in the
// same 16 bytes as an element of the row, so it can be read; blocks without
// one are not), shifted into place in registers, and one 16-byte store a part.
// Measured: 8 x 1025 x 1023 and 2047 x 1025 float32 (105 MB) 20 us, 5.2 TB/s; 16 x
// 1027 x 1020 f16 and 1023 x 1020 (71 MB) 13 us.  (A scalar load an element and
// 64-bit divisions a thread: 25 and 22 us.)
#include "../../include/sgemm_experts.h"
#include "experts.h"
#include "experts_groups.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace {

__device__ __forceinline__ void split_bf16(float x, __nv_bfloat16 (&part)[3]) {
    float rest = x;
    const bool finite = fabsf(x) <= 3.402823466e38f;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        __nv_bfloat16 b = __float2bfloat16_rn(rest);
        if (finite && __hisinf(b)) b = __float2bfloat16_rz(rest);
        part[i] = b;
        rest = finite ? rest - __bfloat162float(b) : 0.f;
    }
}

// Words first .. first + N - 1 of the row at `row` (`bytes` long), from the
// 16-byte blocks that hold them; what lies beyond the row is anything.
template <int N>
__device__ __forceinline__ void load_words(const char* row, long long bytes, int first, uint32_t (&out)[N]) {
    const uintptr_t want = reinterpret_cast<uintptr_t>(row) + 4ull * first;
    const uintptr_t from = want & ~uintptr_t{15}, end = reinterpret_cast<uintptr_t>(row) + bytes;
    constexpr int kWindow = (N + 3 + 3) / 4 * 4;  // N words from any of a block's 4
    uint32_t w[kWindow];
#pragma unroll
    for (int i = 0; i < kWindow; i += 4) {
        uint4 v = {0, 0, 0, 0};
        if (from + 4 * i < end) v = __ldg(reinterpret_cast<const uint4*>(from + 4 * i));
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
    const int shift = static_cast<int>(want >> 2) & 3;
#pragma unroll
    for (int i = 0; i <= N; ++i) w[i] = shift & 2 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = shift & 1 ? w[i + 1] : w[i];
}

template <bool F32>
__device__ __forceinline__ void pack8(const PackJob& j, uint32_t id) {
    const uint32_t octs = (static_cast<uint32_t>(j.cols) + 7) / 8;
    const uint32_t row = id / octs;
    const int c = static_cast<int>(id - row * octs) * 8;
    if (j.offsets) {
        // (boundaries out of order make empty groups too; those are copied)
        const int of = static_cast<int>(row / static_cast<uint32_t>(j.each));
        if (group_bound(j.offsets, of + 1, j.T) <= group_bound(j.offsets, of, j.T)) return;
    }
    uint32_t e = 0, r = row;
    if (j.count > 1) {
        e = row / static_cast<uint32_t>(j.rows);
        r = row - e * static_cast<uint32_t>(j.rows);
    }
    const long long plane = j.count * j.rows * j.dld;
    uint16_t* d = static_cast<uint16_t*>(j.dst) + row * j.dld + c;
    const char* s = static_cast<const char*>(j.src) + (e * j.se + r * j.ld) * (F32 ? 4 : 2);
    const int n = j.cols - c;
    if constexpr (F32) {
        uint32_t x[8];
        load_words<8>(s, 4ll * j.cols, c, x);
        __nv_bfloat16 part[8][3];
#pragma unroll
        for (int i = 0; i < 8; ++i) split_bf16(i < n ? __uint_as_float(x[i]) : 0.f, part[i]);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = __bfloat16_as_ushort(part[2 * i][k]) |
                       static_cast<uint32_t>(__bfloat16_as_ushort(part[2 * i + 1][k])) << 16;
            *reinterpret_cast<uint4*>(d + k * plane) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
        // Rows at odd elements: a word of the copy straddles two of the row's.
        const bool odd = reinterpret_cast<uintptr_t>(s) & 2;
        const char* even = odd ? s - 2 : s;
        uint32_t x[5];
        load_words<5>(even, 2ll * j.cols + (odd ? 2 : 0), c / 2, x);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = odd ? __funnelshift_r(x[i], x[i + 1], 16) : x[i];
            w[i] = 2 * i + 1 < n ? w[i] : 2 * i < n ? w[i] & 0xffffu : 0;
        }
        *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

constexpr int kSteps = 2;

template <bool F32>
__global__ void __launch_bounds__(256) pack_kernel(const PackJob a, const PackJob b, uint32_t na, uint32_t nb) {
    grid_dependency_launch();
    // (CTAs that find nothing to copy cost their start: 4 rows of one of 40 experts of 2047 x 1001 48 us with one step a
    // thread, 32 with two; with four, full copies lose 3 %)
#pragma unroll 1
    for (int u = 0; u < kSteps; ++u) {
        const uint32_t id = (blockIdx.x * kSteps + u) * 256 + threadIdx.x;
        if (id < na)
            pack8<F32>(a, id);
        else if (id - na < nb)
            pack8<F32>(b, id - na);
    }
}

// Matrices that follow one another without a gap are one.
PackJob merged(PackJob j) {
    j.each = j.rows;
    if (j.count > 1 && j.se == j.rows * j.ld) {
        j.rows *= j.count;
        j.count = 1;
    }
    return j;
}

}  // namespace

int experts_pack(const PackJob& a, const PackJob& b, bool f32, cudaStream_t s) {
    const long long na = a.dst ? a.count * a.rows * ((a.cols + 7) / 8) : 0;
    const long long nb = b.dst ? b.count * b.rows * ((b.cols + 7) / 8) : 0;
    if (na + nb == 0) return SGEMM_OK;
    if (na + nb > 0xffffff00ll) return SGEMM_ERR_INVALID_ARG;  // (2^35 elements: 64 GB of 16-bit ones)
    const unsigned ctas = static_cast<unsigned>((na + nb + 256 * kSteps - 1) / (256 * kSteps));
    const PackJob ja = merged(a), jb = merged(b);
    if (f32)
        pack_kernel<true><<<ctas, 256, 0, s>>>(ja, jb, static_cast<uint32_t>(na), static_cast<uint32_t>(nb));
    else
        pack_kernel<false><<<ctas, 256, 0, s>>>(ja, jb, static_cast<uint32_t>(na), static_cast<uint32_t>(nb));
    return cudaGetLastError() == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}

}  // namespace gb300
