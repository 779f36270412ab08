// Launches of the tensor-core grouped products (experts_tc.cuh): operand
// copies where needed, tensor maps, tile shape and grid.
#include "../../include/sgemm_experts.h"
#include "experts_tc.cuh"

#include "api_internal.h"
#include "experts.h"

namespace gb300 {
namespace detail {
namespace {

// Rows an expert on average up to which float32 products run on the CUDA cores
// (experts_few.cu).  Measured for 8 experts of 1024 x 2048, us there (by parts 50):
// 4 13, 8 19, 16 26, 18 49 (transposed 14, 21, 44, 57); for 64 experts of that size (by
// parts 353): 8 130, 12 199, 18 281 (transposed 189, 307, 442).  Uneven groups take
// less there, not more: the same 18 on average with a fifth of all rows in one
// expert 244, all in one 194 (transposed 390, 309): a long group's tiles share
// their weights.
constexpr long long kFewRows = 18;

// An operand as the tensor maps read it: 16-bit elements, third dimension the
// matrices (and planes of parts).
struct TcOperand {
    const void* p;
    long long inner, rows, third, ld, stride;  // elements
};

int encode_3d(CUtensorMap* map, const TcOperand& o, bool f16, int box_inner, int box_rows) {
    if (!g_encode) return SGEMM_ERR_CUDA;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(o.inner), static_cast<cuuint64_t>(o.rows),
                                static_cast<cuuint64_t>(o.third)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(o.ld) * 2, static_cast<cuuint64_t>(o.stride) * 2};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r =
        g_encode(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                 const_cast<void*>(o.p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                 CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SGEMM_OK : SGEMM_ERR_CUDA;
}

// 16-bit matrices that a tensor map reads as they are.
bool tma_readable(const MatrixArg& m) {
    return (reinterpret_cast<uintptr_t>(m.p) & 15) == 0 && (m.rows == 1 || m.ld % 8 == 0) &&
           (m.count == 1 || m.se % 8 == 0);
}

template <bool AMN, bool BMN, int TN, int CG, int PARTS, bool SPLIT = false>
int launch(const CUtensorMap& a, const CUtensorMap& b, const GroupedTcParams& p, long long tiles,
           const DeviceState& st, cudaStream_t s) {
    using S = GroupedShape<TN, CG, PARTS>;
    const auto kernel = grouped_tc_kernel<AMN, BMN, TN, CG, PARTS, SPLIT>;
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
    if (cudaLaunchKernelEx(&cfg, kernel, a, b, p) != cudaSuccess) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

struct Tile {
    int tn, cg;  // columns; CTAs that share a tile
};

// Tile of a product.  Measured on GB300, bf16, us for 128 columns a CTA / 128 a
// pair / 256 a pair, by rows an expert on average (16 experts of 2048 x 2048):
// 16 23.6 / 24.5 / 24.6, 64 24.2 / 25.3 / 26.3, 96 25.3 / 26.2 / 26.8, 128 29.4 /
// 29.0 / 27.3, 256 40.1 / 37.6 / 35.1, 512 57.5 / 52.6 / 53.5; 8 experts of 4096
// x 1024: 96 15.5 / 14.3 / 20.0, 256 26.8 / 26.8 / 24.5, 512 31.2 / 29.3 / 43.4.
// So: single CTAs up to 96 rows an expert (the weights' bytes count, and more,
// smaller tiles spread them more evenly), else pairs, with the width whose
// rounds of tiles over the GPU come to fewer columns; half the width moves A
// twice as often and has to save a quarter (16 experts of 4096 x 4096 and 16384
// rows: 320 us for a pair's 128 columns, 293 for 256).  float32, whose stages
// hold three parts of either operand, has 128 (64: 45 us instead of 39 for 2047
// rows, 8 experts of 1025 x 1023, although that is two rounds of tiles).
Tile choose_tile(const GroupedCall& c, const DeviceState& st) {
    if (c.type == SGEMM_TYPE_F32) return {128, 2};
    const long long groups = std::min(c.T, c.E);
    if (!c.wgrad && c.T <= 96 * groups) return {128, 1};
    const long long ft = ceil_div(c.F, 256);
    auto columns = [&](int tn) {  // of one pair, over its rounds
        const long long t = c.wgrad ? c.E * ceil_div(c.C, tn) : ceil_div(c.T, tn) + groups / 2;
        return ceil_div(t * ft, st.max_pairs) * tn;
    };
    return {columns(128) * 13 < columns(256) * 10 ? 128 : 256, 2};
}

template <bool AMN, bool BMN, int TN, int CG, int PARTS, bool SPLIT = false>
int set_up() {
    return cudaFuncSetAttribute(grouped_tc_kernel<AMN, BMN, TN, CG, PARTS, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                GroupedShape<TN, CG, PARTS>::kSmem) == cudaSuccess
               ? SGEMM_OK
               : SGEMM_ERR_CUDA;
}

template <bool AMN>
int launch_forward(const Tile& tile, bool f32, const CUtensorMap& a, const CUtensorMap& b, const GroupedTcParams& p,
                   long long tiles, const DeviceState& st, cudaStream_t s) {
    if (f32) return launch<AMN, false, 128, 2, 3>(a, b, p, tiles, st, s);
    if (tile.cg == 1)
        return p.ks > 1 ? launch<AMN, false, 128, 1, 1, true>(a, b, p, tiles, st, s)
                        : launch<AMN, false, 128, 1, 1>(a, b, p, tiles, st, s);
    return tile.tn == 128 ? launch<AMN, false, 128, 2, 1>(a, b, p, tiles, st, s)
                          : launch<AMN, false, 256, 2, 1>(a, b, p, tiles, st, s);
}

// Operands of one product copied into the library's pool for the length of
// the call.
struct Packs {
    void* ws = nullptr;
    cudaStream_t s = nullptr;
    ~Packs() {
        if (ws) (void)cudaFreeAsync(ws, s);
    }
};

}  // namespace

int experts_tc_set_up(DeviceState& st) {
    if (set_up<true, false, 128, 1, 1, true>() || set_up<false, false, 128, 1, 1, true>() ||
        set_up<true, false, 128, 1, 1>() || set_up<true, false, 128, 2, 1>() || set_up<true, false, 256, 2, 1>() ||
        set_up<false, false, 128, 1, 1>() || set_up<false, false, 128, 2, 1>() || set_up<false, false, 256, 2, 1>() ||
        set_up<true, true, 128, 2, 1>() || set_up<true, true, 256, 2, 1>() || set_up<true, false, 128, 2, 3>() ||
        set_up<false, false, 128, 2, 3>() || set_up<true, true, 128, 2, 3>()) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    // Pairs that fit the GPU at once: persistent kernels launch no more.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * st.sm_count);
    cfg.blockDim = dim3(GroupedShape<256, 2, 1>::kThreads);
    cfg.dynamicSmemBytes = GroupedShape<256, 2, 1>::kSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&st.max_pairs, grouped_tc_kernel<true, false, 256, 2, 1>, &cfg) !=
            cudaSuccess ||
        st.max_pairs < 1) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

int grouped_tc(const GroupedCall& c, int dev, DeviceState& st, cudaStream_t s) {
    // (float32 with few rows an expert; where its grid would be too large, the parts)
    if (c.type == SGEMM_TYPE_F32 && !c.wgrad && c.T <= kFewRows * std::min(c.T, c.E)) {
        const int rc = grouped_few(c, st, s);
        if (rc != SGEMM_ERR_UNSUPPORTED) return rc;
    }
    const bool f32 = c.type == SGEMM_TYPE_F32, f16 = c.type == SGEMM_TYPE_F16;
    // The first dimension of every operand as stored: A (W, or X) and B (X, or dY).
    const MatrixArg m[2] = {c.a, c.b};
    TcOperand o[2];
    PackJob job[2] = {};
    size_t bytes[2] = {0, 0};
    for (int i = 0; i < 2; ++i) {
        const bool copy = f32 || !tma_readable(m[i]);
        const long long dld = (m[i].cols + 7) / 8 * 8;
        if (copy) {
            job[i] = {m[i].p, m[i].count, m[i].rows, m[i].ld, m[i].se, static_cast<int>(m[i].cols), nullptr, dld,
                      i == 0 && !c.wgrad ? c.offsets : nullptr, c.T, 0};
            bytes[i] = (static_cast<size_t>(f32 ? 3 : 1) * m[i].count * m[i].rows * dld * 2 + 255) & ~size_t{255};
            o[i] = {nullptr, m[i].cols, m[i].rows, (f32 ? 3 : 1) * m[i].count, dld, m[i].rows * dld};
        } else {
            // (a dimension of one row or matrix has no stride of its own: any that the encoder takes)
            const long long ld = m[i].rows > 1 ? m[i].ld : dld;
            o[i] = {m[i].p, m[i].cols, m[i].rows, m[i].count, ld, m[i].count > 1 ? m[i].se : m[i].rows * ld};
        }
    }
    Packs packs;
    packs.s = s;
    if (bytes[0] + bytes[1]) {
        cudaMemPool_t pool = workspace_pool(dev, st);
        if (!pool || cudaMallocFromPoolAsync(&packs.ws, bytes[0] + bytes[1], pool, s) != cudaSuccess) {
            (void)cudaGetLastError();
            packs.ws = nullptr;
            return SGEMM_ERR_CUDA;
        }
        if (bytes[0]) o[0].p = job[0].dst = packs.ws;
        if (bytes[1]) o[1].p = job[1].dst = static_cast<char*>(packs.ws) + bytes[0];
        const int rc = experts_pack(job[0], job[1], f32, s);
        if (rc != SGEMM_OK) return rc;
    }

    const Tile tile = choose_tile(c, st);
    const int tn = tile.tn, cg = tile.cg;
    GroupedTcParams p = {};
    p.offsets = c.offsets;
    p.T = c.T, p.E = c.E;
    p.F = c.F, p.C = c.C, p.K = c.K;
    p.ftiles = static_cast<int>(ceil_div(c.F, 128 * cg));
    p.ctiles = c.wgrad ? static_cast<int>(ceil_div(c.C, tn)) : 0;
    p.a_planes = c.wgrad ? 1 : c.E;
    p.out = c.out, p.ldo = c.ldo, p.so = c.so, p.out_type = c.out_type;
    p.align = row_alignment(c.out, c.out_type == SGEMM_TYPE_F32 ? 4 : 2, c.ldo, c.so);
    p.timeout_ns = kDefaultTimeoutNs;
    p.status = st.status_word;
    const uint32_t fmt = f16 ? 0 : 1;
    p.idesc = 1u << 4 | fmt << 7 | fmt << 10 | (c.a_mn ? 1u << 15 : 0) | (c.wgrad ? 1u << 16 : 0) |
              static_cast<uint32_t>(128 * cg / 16) << 24;
    const long long tiles = c.wgrad ? static_cast<long long>(c.E) * p.ftiles * p.ctiles
                                    : (c.T / tn + std::min(c.T, c.E)) * static_cast<long long>(p.ftiles);
    if (tiles > 0x7fffffffll - 65536) return SGEMM_ERR_INVALID_ARG;
    p.ks = cg == 1 ? split_parts(tiles, c.K, 256, st.sm_count) : 1;
    alignas(64) CUtensorMap ma, mb;
    int rc = encode_3d(&ma, o[0], f16, 64, c.a_mn ? 64 : 128);
    if (rc == SGEMM_OK) rc = encode_3d(&mb, o[1], f16, 64, std::min(64, tn / cg));
    if (rc != SGEMM_OK) return rc;
    if (c.wgrad)
        return f32         ? launch<true, true, 128, 2, 3>(ma, mb, p, tiles, st, s)
               : tn == 128 ? launch<true, true, 128, 2, 1>(ma, mb, p, tiles, st, s)
                           : launch<true, true, 256, 2, 1>(ma, mb, p, tiles, st, s);
    return c.a_mn ? launch_forward<true>(tile, f32, ma, mb, p, tiles, st, s)
                  : launch_forward<false>(tile, f32, ma, mb, p, tiles, st, s);
}

}  // namespace detail
}  // namespace gb300
