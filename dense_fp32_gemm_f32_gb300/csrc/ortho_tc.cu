// Launches of an orthogonalised update: the workspace's parts, tensor maps, tile
// shape (ortho_tc.cuh).
#include "../../include/sgemm_ortho.h"
#include "ortho_tc.cuh"

#include "api_internal.h"
#include "ortho.h"

namespace gb300 {
namespace detail {
namespace {

// f16 planes of E matrices of rows x inner, `pitch` elements a row, as the
// tensor maps read them: boxes of 64 x 64.
int encode_planes(CUtensorMap* map, const void* p, long long inner, long long rows, long long planes, long long pitch) {
    if (!g_encode) return SGEMM_ERR_CUDA;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(planes)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch) * 2, static_cast<cuuint64_t>(pitch * rows) * 2};
    const cuuint32_t box[3] = {64, 64, 1}, ones[3] = {1, 1, 1};
    const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p), dims, strides, box, ones,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SGEMM_OK : SGEMM_ERR_CUDA;
}

template <int TN, int PARTS, bool TALL>
int set_up() {
    return cudaFuncSetAttribute(ortho_tc_kernel<TN, PARTS, TALL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                OrthoShape<TN, PARTS>::kSmem) == cudaSuccess
               ? SGEMM_OK
               : SGEMM_ERR_CUDA;
}

template <int TN, int PARTS>
int set_up_both() {
    return set_up<TN, PARTS, false>() || set_up<TN, PARTS, true>();
}

int set_up_kernels() {
    if (set_up_both<256, 1>() || set_up_both<128, 1>() || set_up_both<64, 1>() || set_up_both<128, 2>() ||
        set_up_both<64, 2>()) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

template <int TN, int PARTS>
int launch(OrthoTcParams& p, const CUtensorMap (&maps)[4], const DeviceState& st, cudaStream_t s) {
    using S = OrthoShape<TN, PARTS>;
    const bool tall = p.rows > p.cols;
    const long long ft = ceil_div(p.m, S::FT), ct = ceil_div(p.m, TN);
    long long sym = ft * ct;
    p.mirror = p.E * sym > st.max_pairs || ft > 32;
    if (p.mirror) {
        sym = 0;
        for (long long f = 0; f < ft; ++f) sym += std::min(ct, (f + 1) * S::R);
    }
    const long long up = ceil_div(p.rows, S::FT) * ceil_div(p.cols, TN), most = p.E * std::max(sym, up);
    const long long items = p.steps * p.E * (2 * sym + up);
    if (items > 0x7fffffffll - 65536) return SGEMM_ERR_INVALID_ARG;
    p.sym_tiles = static_cast<int>(sym), p.up_tiles = static_cast<int>(up), p.items = static_cast<int>(items);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<long long>(most, st.max_pairs)));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;  // tiles wait for those of other CTAs
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const auto kernel = tall ? ortho_tc_kernel<TN, PARTS, true> : ortho_tc_kernel<TN, PARTS, false>;
    if (cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], maps[3], p) != cudaSuccess) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

}  // namespace

OrthoLayout ortho_layout(int E, int M, int N, int steps, int parts) {
    const long long m = std::min(M, N);
    OrthoLayout l = {};
    l.pitch = (N + 15ll) / 16 * 16, l.square_pitch = (m + 15) / 16 * 16;  // (the epilogue's accesses of 32 bytes)
    // Row chunks of about 8192 elements, a few rounds of the GPU at most.
    l.chunks = static_cast<int>(std::max(1ll, std::min({static_cast<long long>(kOrthoMostChunks), static_cast<long long>(M),
                                                        M * l.pitch / 8192})));
    l.per = static_cast<int>(ceil_div(M, l.chunks));
    l.chunks = static_cast<int>(ceil_div(M, l.per));
    l.panels = static_cast<int>(ceil_div(m, 256));
    auto take = [&](long long bytes) {
        const long long at = l.bytes;
        l.bytes += (bytes + 255) / 256 * 256;
        return at;
    };
    l.part = take(8ll * E * l.chunks);
    l.done = take(4ll * 3 * E * l.panels);
    l.shift = take(4ll * E);
    l.d = take(4ll * E * l.square_pitch);
    l.e = take(4ll * E * l.square_pitch);
    l.a = take(2ll * 2 * E * m * l.square_pitch);
    l.p = take(2ll * parts * E * m * l.square_pitch);  // (with one plane products take B's hi alone)
    l.x[0] = take(2ll * 2 * E * M * l.pitch);
    l.x[1] = steps > 1 ? take(2ll * 2 * E * M * l.pitch) : l.x[0];
    return l;
}

int orthogonalize(const OrthoCall& c, DeviceState& st, cudaStream_t s) {
    std::call_once(st.ortho_once, [&] {
        st.ortho_status = set_up_kernels() != SGEMM_OK ? SGEMM_ERR_CUDA : ortho_small_set_up(&st.ortho_ctas);
    });
    if (st.ortho_status != SGEMM_OK) return st.ortho_status;
    if (const int rc = ortho_small(c, st, s); rc != SGEMM_ERR_UNSUPPORTED) return rc;
    const int m = std::min(c.M, c.N), parts = c.parts;
    const OrthoLayout l = ortho_layout(c.E, c.M, c.N, c.steps, parts);
    if (static_cast<long long>(c.E) * l.chunks > 0x7fffffffll) return SGEMM_ERR_INVALID_ARG;
    char* const ws = static_cast<char*>(c.workspace);
    auto planes = [&](long long at, long long ld, long long matrix) {
        __half* const hi = reinterpret_cast<__half*>(ws + at);
        return OrthoPlanes{hi, hi + c.E * matrix, ld, matrix};
    };
    OrthoPrep prep = {};
    prep.chunks = l.chunks, prep.per = l.per;
    OrthoTcParams p = {};
    p.E = c.E, p.m = m, p.rows = c.M, p.cols = c.N, p.steps = c.steps;
    prep.part = reinterpret_cast<double*>(ws + l.part);
    prep.zero = p.done = reinterpret_cast<int*>(ws + l.done);
    prep.zeros = 3ll * c.E * l.panels;
    p.panels = l.panels;
    prep.shift = reinterpret_cast<int*>(ws + l.shift);
    p.shift = prep.shift, p.growth = c.growth;
    p.d = reinterpret_cast<float*>(ws + l.d);
    p.e = reinterpret_cast<float*>(ws + l.e);
    p.diag = l.square_pitch;
    p.a = planes(l.a, l.square_pitch, m * l.square_pitch);
    p.p = planes(l.p, l.square_pitch, m * l.square_pitch);
    for (int i = 0; i < 2; ++i) p.x[i] = planes(l.x[i], l.pitch, c.M * l.pitch);
    p.c1 = c.a, p.c3 = c.b, p.c5 = c.c;
    p.out = c.out, p.ldo = c.ldo, p.so = c.so, p.out_type = c.type;
    p.align = row_alignment(c.out, c.type == SGEMM_TYPE_F32 ? 4 : 2, c.M > 1 ? c.ldo : 0, c.E > 1 ? c.so : 0);
    p.timeout_ns = kDefaultTimeoutNs;
    p.status = st.status_word;
    alignas(64) CUtensorMap maps[4];
    const OrthoPlanes* const of[4] = {&p.x[0], &p.x[1], &p.a, &p.p};
    for (int i = 0; i < 4; ++i) {
        const long long count = (i < 3 ? 2ll : parts) * c.E;
        const int rc = i < 2 ? encode_planes(&maps[i], of[i]->hi, c.N, c.M, count, l.pitch)
                             : encode_planes(&maps[i], of[i]->hi, m, m, count, l.square_pitch);
        if (rc != SGEMM_OK) return rc;
    }
    prep.G = c.G, prep.ldg = c.ldg, prep.sg = c.sg;
    prep.E = c.E, prep.rows = c.M, prep.cols = c.N;
    prep.vec = row_alignment(c.G, c.type == SGEMM_TYPE_F32 ? 4 : 2, c.M > 1 ? c.ldg : 0, c.E > 1 ? c.sg : 0) == 16;
    prep.eps = c.eps;
    prep.hi = reinterpret_cast<uint16_t*>(p.x[0].hi), prep.pitch = l.pitch, prep.plane = c.E * p.x[0].matrix;
    const int rc = ortho_prepare(prep, c.type, s);
    if (rc != SGEMM_OK) return rc;
    // Tiles of a pair of CTAs: 256 rows by 128 columns; with one plane 256 where the GPU's pairs then have two and a half each in an update.
    // Measured, us for 256 columns / 128 / single CTAs with 128 x 128 (one plane): 512 x 512 173 / 110 / 112, 1024 x 1024
    // 213 / 135 / 136, 8 of 200 x 4000 232 / 186 / 198, 2048 x 4096 406 / 338 / 354 (128 tiles of 256 columns, 76 pairs),
    // 2 of 3000 x 3000 (288) 768 / 897 / 942.  Two planes of either operand (float32), 128 columns of a pair / single
    // CTAs: 200 x 300 122 / 125, 2048 x 2048 420 / 445, 2 of 3000 x 3000 2178 / 2492.
    // 64 columns where there are few tiles: each is done sooner, and its epilogue has registers enough. us for 64 columns / 128, two planes:
    // 129 x 129 75 / 105, 1024 x 1024 (64 tiles of 64 columns) 139 / 193, 2 of 1024 x 1024 (128) 177 / 199, 2 of 1025 x 1023 (160) 205 / 219,
    // 3 of 1024 x 1024 (192) 221 / 255, 4 of them (256) 269 / 261, 2048 x 2048 (256) 467 / 402; one plane: 300 x 700 (22) 79 / 98, 1024 x 1024
    // 99 / 119, 1152 x 1152 (90) 128 / 124, 1500 x 1500 (144) 173 / 149.
    const long long narrow = c.E * ceil_div(c.M, 256) * ceil_div(c.N, 64);
    if (narrow <= (parts == 2 ? 8ll * st.max_pairs / 3 : st.max_pairs))
        return parts == 2 ? launch<64, 2>(p, maps, st, s) : launch<64, 1>(p, maps, st, s);
    if (parts == 2) return launch<128, 2>(p, maps, st, s);
    const long long tiles = c.E * ceil_div(c.M, 256) * ceil_div(c.N, 256);
    return 2 * tiles >= 5 * st.max_pairs ? launch<256, 1>(p, maps, st, s) : launch<128, 1>(p, maps, st, s);
}

}  // namespace detail
}  // namespace gb300
