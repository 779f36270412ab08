// Launches of the MXFP4 products (mxfp4_tc.cuh): tensor maps, tile and grid.
#include "mxfp4_tc.cuh"

#include "../../include/sgemm_experts.h"
#include "api_internal.h"
#include "experts.h"

namespace gb300 {
namespace detail {
namespace {

int encode_bytes(CUtensorMap* map, const void* p, CUtensorMapDataType type, int size, long long inner, long long rows,
                 long long third, int box_inner, int box_rows, CUtensorMapSwizzle swizzle) {
    if (!g_encode) return SGEMM_ERR_CUDA;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(third)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(inner * size), static_cast<cuuint64_t>(rows * inner * size)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r = g_encode(map, type, 3, const_cast<void*>(p), dims, strides, box, ones,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SGEMM_OK : SGEMM_ERR_CUDA;
}

template <int TN, int CG, bool SPLIT = false, bool LONG = false>
int launch(const CUtensorMap (&m)[4], const Mxfp4TcParams& p, long long tiles, const DeviceState& st,
           cudaStream_t s) {
    using S = Mxfp4Shape<TN, CG, LONG>;
    const int share = SPLIT ? p.ks : CG;  // CTAs of a cluster
    cudaLaunchConfig_t cfg = {};
    // (a pair's tiles may be split into columns of 64: LastRound)
    cfg.gridDim = dim3(static_cast<unsigned>(CG == 2 ? 2 * std::min<long long>(tiles * (TN / 64), st.max_pairs)
                                                     : SPLIT ? tiles * p.ks : std::min<long long>(tiles, st.sm_count)));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    // The kernel's set-up may run beside the end of the kernel before it (the
    // quantiser, the operand copies): it reads global memory only after it has
    // waited for that one.
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(share);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = share > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, mxfp4_tc_kernel<TN, CG, SPLIT, LONG>, m[0], m[1], m[2], m[3], p) != cudaSuccess) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

template <int TN, int CG, bool SPLIT = false, bool LONG = false>
int set_up() {
    return cudaFuncSetAttribute(mxfp4_tc_kernel<TN, CG, SPLIT, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Mxfp4Shape<TN, CG, LONG>::kSmem) == cudaSuccess
               ? SGEMM_OK
               : SGEMM_ERR_CUDA;
}

}  // namespace

int mxfp4_tc_set_up() {
    if (set_up<64, 1, true>() || set_up<64, 1>() || set_up<192, 2>() || set_up<64, 1, true, true>() ||
        set_up<64, 1, false, true>() || set_up<192, 2, false, true>()) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

int mxfp4_tc(const Mxfp4Call& c, const DeviceState& st, cudaStream_t s) {
    const bool narrow = c.T <= 64ll * std::min(c.T, c.E);
    const int tn = narrow ? 64 : 192, cg = narrow ? 1 : 2;
    const long long kb = ceil_div(c.K, 32), kq = ceil_div(c.K, 128);
    Mxfp4TcParams p = {};
    p.offsets = c.offsets;
    p.T = c.T, p.E = c.E, p.F = c.N, p.K = static_cast<int>(32 * kb);
    p.ftiles = static_cast<int>(ceil_div(c.N, 128 * cg));
    p.out = c.out, p.ldo = c.ldo, p.out_type = c.out_type;
    p.align = row_alignment(c.out, c.out_type == SGEMM_TYPE_F32 ? 4 : 2, c.ldo, 0);
    p.timeout_ns = kDefaultTimeoutNs;
    p.status = st.status_word;
    const long long tiles = (c.T / tn + std::min(c.T, c.E)) * static_cast<long long>(p.ftiles);
    if (tiles > 0x7fffffffll - 65536) return SGEMM_ERR_INVALID_ARG;
    alignas(64) CUtensorMap m[4];
    int rc = encode_bytes(&m[0], c.W, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 16 * kb, c.N, c.E, 128, 128,
                          CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc == SGEMM_OK)
        rc = encode_bytes(&m[1], c.X, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 16 * kb, c.T, 1, 128,
                          narrow ? Mxfp4Shape<64, 1>::kBoxCols : Mxfp4Shape<192, 2>::kBoxCols,
                          CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc == SGEMM_OK)
        rc = encode_bytes(&m[2], c.w_scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, 128 * kq, ceil_div(c.N, 128), c.E, 256,
                          1, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc == SGEMM_OK)
        rc = encode_bytes(&m[3], c.x_scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, 128 * kq, c.x_blocks, 1, 256,
                          narrow ? Mxfp4Shape<64, 1>::kSbBlocks : Mxfp4Shape<192, 2>::kSbBlocks, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc != SGEMM_OK) return rc;
    p.ks = narrow ? split_parts(tiles, p.K, 1024, st.sm_count) : 1;
    if (p.K > static_cast<long long>(kMxChunk) * p.ks) {  // (of a cluster's part)
        if (p.ks > 1) return launch<64, 1, true, true>(m, p, tiles, st, s);
        return narrow ? launch<64, 1, false, true>(m, p, tiles, st, s) : launch<192, 2, false, true>(m, p, tiles, st, s);
    }
    if (p.ks > 1) return launch<64, 1, true>(m, p, tiles, st, s);
    return narrow ? launch<64, 1>(m, p, tiles, st, s) : launch<192, 2>(m, p, tiles, st, s);
}

}  // namespace detail
}  // namespace gb300
