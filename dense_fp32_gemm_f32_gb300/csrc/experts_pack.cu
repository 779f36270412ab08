// Copies of operands that the tensor maps cannot read: 16-bit rows off the
// 16-byte grid into pitched rows, and float32 operands into three bf16 parts,
//     x0 = bf16(x), x1 = bf16(x - x0), x2 = bf16(x - x0 - x1),
// each difference exact in float32 (x's 24 bits less the 8 leading ones of
// what is left, twice), so that what the parts miss is below 2^-25 |x|.  A
// finite x that bf16 would round to infinity is cut instead; the parts of a
// non-finite x are x, 0, 0.
//
// Bound by bytes: 4 read and 6 written a float32.  A thread takes 4
// neighbouring elements: one 16-byte load where the row allows it, an 8-byte
// store a part.
#include "../../include/sgemm_experts.h"
#include "experts.h"
#include "experts_groups.cuh"

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

__device__ __forceinline__ void pack_row4(const PackJob& j, long long id, bool f32) {
    const long long quads = (j.cols + 3) / 4;
    const long long row = id / quads;
    const int c = static_cast<int>(id % quads) * 4;
    const long long e = row / j.rows, r = row % j.rows;
    const long long plane = j.count * j.rows * j.dld;
    uint16_t* d = static_cast<uint16_t*>(j.dst) + row * j.dld + c;
    const int n = j.cols - c;
    if (f32) {
        const float* s = static_cast<const float*>(j.src) + e * j.se + r * j.ld + c;
        float x[4];
        if (n >= 4 && (reinterpret_cast<uintptr_t>(s) & 15) == 0) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(s));
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = i < n ? s[i] : 0.f;
        }
        __nv_bfloat16 part[4][3];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_bf16(x[i], part[i]);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            uint2 w;
            w.x = __bfloat16_as_ushort(part[0][k]) | static_cast<uint32_t>(__bfloat16_as_ushort(part[1][k])) << 16;
            w.y = __bfloat16_as_ushort(part[2][k]) | static_cast<uint32_t>(__bfloat16_as_ushort(part[3][k])) << 16;
            *reinterpret_cast<uint2*>(d + k * plane) = w;
        }
    } else {
        const uint16_t* s = static_cast<const uint16_t*>(j.src) + e * j.se + r * j.ld + c;
        uint16_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = i < n ? s[i] : 0;
        uint2 w;
        w.x = x[0] | static_cast<uint32_t>(x[1]) << 16;
        w.y = x[2] | static_cast<uint32_t>(x[3]) << 16;
        *reinterpret_cast<uint2*>(d) = w;
    }
}

__global__ void __launch_bounds__(256) pack_kernel(const PackJob a, const PackJob b, long long na, long long nb,
                                                   bool f32) {
    const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (id < na)
        pack_row4(a, id, f32);
    else if (id < na + nb)
        pack_row4(b, id - na, f32);
}

}  // namespace

int experts_pack(const PackJob& a, const PackJob& b, bool f32, cudaStream_t s) {
    const long long na = a.dst ? a.count * a.rows * ((a.cols + 3) / 4) : 0;
    const long long nb = b.dst ? b.count * b.rows * ((b.cols + 3) / 4) : 0;
    const long long ctas = (na + nb + 255) / 256;
    if (ctas == 0) return SGEMM_OK;
    if (ctas > 0x7fffffffll) return SGEMM_ERR_INVALID_ARG;
    pack_kernel<<<static_cast<unsigned>(ctas), 256, 0, s>>>(a, b, na, nb, f32);
    return cudaGetLastError() == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}

}  // namespace gb300
