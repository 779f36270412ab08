// Launches of an orthogonalised update: workspace, tensor maps, tile shape, and
// the three products of every step (ortho_tc.cuh).
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

template <int MODE, bool AMN, bool BMN, int TN, int CG, int PARTS>
int set_up() {
    return cudaFuncSetAttribute(ortho_tc_kernel<MODE, AMN, BMN, TN, CG, PARTS>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                OrthoShape<TN, CG, PARTS>::kSmem) == cudaSuccess
               ? SGEMM_OK
               : SGEMM_ERR_CUDA;
}

template <int TN, int CG, int PARTS>
int set_up_all() {
    return set_up<kOrthoGram, false, false, TN, CG, PARTS>() || set_up<kOrthoGram, true, true, TN, CG, PARTS>() ||
           set_up<kOrthoSquare, false, false, TN, CG, PARTS>() || set_up<kOrthoUpdate, false, true, TN, CG, PARTS>() ||
           set_up<kOrthoUpdate, false, false, TN, CG, PARTS>();
}

template <int MODE, bool AMN, bool BMN, int TN, int CG, int PARTS>
int launch(const CUtensorMap& a, const CUtensorMap& b, OrthoTcParams p, const DeviceState& st, cudaStream_t s) {
    constexpr int FT = 128 * CG;
    p.ftiles = static_cast<int>(ceil_div(p.F, FT));
    p.ctiles = static_cast<int>(ceil_div(p.C, TN));
    long long per = static_cast<long long>(p.ftiles) * p.ctiles;
    if (MODE != kOrthoUpdate) {
        per = 0;
        for (int f = 0; f < p.ftiles; ++f) per += std::min(p.ctiles, (f + 1) * (FT / TN));
    }
    if (per * p.E > 0x7fffffffll - 65536) return SGEMM_ERR_INVALID_ARG;
    p.per = static_cast<int>(per);
    p.tiles = p.per * p.E;
    p.idesc = 1u << 4 | (AMN ? 1u << 15 : 0) | (BMN ? 1u << 16 : 0) | static_cast<uint32_t>(TN / 8) << 17 |
              static_cast<uint32_t>(FT / 16) << 24;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(CG == 2 ? 2 * std::min(p.tiles, st.max_pairs) : std::min(p.tiles, st.sm_count)));
    cfg.blockDim = dim3(OrthoShape<TN, CG, PARTS>::kThreads);
    cfg.dynamicSmemBytes = OrthoShape<TN, CG, PARTS>::kSmem;
    cfg.stream = s;
    // (the kernel's set-up may run beside the end of the one before it)
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, ortho_tc_kernel<MODE, AMN, BMN, TN, CG, PARTS>, a, b, p) != cudaSuccess) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

int set_up_kernels() {
    if (set_up_all<256, 2, 1>() || set_up_all<128, 1, 1>() || set_up_all<128, 2, 2>() || set_up_all<128, 1, 2>()) {
        (void)cudaGetLastError();
        return SGEMM_ERR_CUDA;
    }
    return SGEMM_OK;
}

struct Workspace {
    void* p = nullptr;
    cudaStream_t s = nullptr;
    ~Workspace() {
        if (p) (void)cudaFreeAsync(p, s);
    }
};

template <int TN, int CG, int PARTS>
int steps(const OrthoCall& c, const OrthoPrep& prep, char* const (&x)[2], char* a, char* b, float* d, float* e,
          const DeviceState& st, cudaStream_t s) {
    const bool tall = c.M > c.N;
    const int m = std::min(c.M, c.N), n = std::max(c.M, c.N);
    const long long mp = (m + 15) / 16 * 16, xs = static_cast<long long>(c.M) * prep.pitch, ms = m * mp;
    alignas(64) CUtensorMap tx[2], ta, tb;
    for (int i = 0; i < 2; ++i)
        if (const int rc = encode_planes(&tx[i], x[i], c.N, c.M, 2ll * c.E, prep.pitch)) return rc;
    if (const int rc = encode_planes(&ta, a, m, m, 2ll * c.E, mp)) return rc;
    if (const int rc = encode_planes(&tb, b, m, m, static_cast<long long>(PARTS) * c.E, mp)) return rc;
    OrthoTcParams p = {};
    p.E = c.E, p.diag = mp;
    p.a = c.a, p.b = c.b, p.c = c.c;
    p.timeout_ns = kDefaultTimeoutNs;
    p.status = st.status_word;
    auto plane = [](char* q, int i, long long size) { return reinterpret_cast<__half*>(q) + i * size; };
    for (int step = 0; step < c.steps; ++step) {
        const int from = step & 1, to = from ^ 1;
        OrthoTcParams g = p;
        g.F = g.C = m, g.K = n;
        g.out_hi = plane(a, 0, c.E * ms), g.out_lo = plane(a, 1, c.E * ms);
        g.ld_out = mp, g.s_out = ms, g.d_out = d;
        int rc = tall ? launch<kOrthoGram, true, true, TN, CG, PARTS>(tx[from], tx[from], g, st, s)
                      : launch<kOrthoGram, false, false, TN, CG, PARTS>(tx[from], tx[from], g, st, s);
        if (rc != SGEMM_OK) return rc;
        OrthoTcParams q = p;
        q.F = q.C = q.K = m;
        q.in_hi = g.out_hi, q.in_lo = g.out_lo, q.ld_in = mp, q.s_in = ms, q.d_in = d;
        q.out_hi = plane(b, 0, c.E * ms), q.out_lo = PARTS == 2 ? plane(b, 1, c.E * ms) : nullptr;
        q.ld_out = mp, q.s_out = ms, q.d_out = e;
        rc = launch<kOrthoSquare, false, false, TN, CG, PARTS>(ta, ta, q, st, s);
        if (rc != SGEMM_OK) return rc;
        OrthoTcParams u = p;
        u.F = c.M, u.C = c.N, u.K = m;
        u.in_hi = plane(x[from], 0, c.E * xs), u.in_lo = plane(x[from], 1, c.E * xs), u.ld_in = prep.pitch, u.s_in = xs;
        u.d_in = e, u.by_column = tall;
        if (step + 1 < c.steps) {
            u.out_hi = plane(x[to], 0, c.E * xs), u.out_lo = plane(x[to], 1, c.E * xs);
            u.ld_out = prep.pitch, u.s_out = xs;
        } else {
            u.out = c.out, u.ldo = c.ldo, u.so = c.so, u.out_type = c.type;
            u.align = row_alignment(c.out, c.type == SGEMM_TYPE_F32 ? 4 : 2, c.M > 1 ? c.ldo : 0, c.E > 1 ? c.so : 0);
        }
        // X' = P X; tall, X^T stored: X'^T = X^T P.
        rc = tall ? launch<kOrthoUpdate, false, false, TN, CG, PARTS>(tx[from], tb, u, st, s)
                  : launch<kOrthoUpdate, false, true, TN, CG, PARTS>(tb, tx[from], u, st, s);
        if (rc != SGEMM_OK) return rc;
    }
    return SGEMM_OK;
}

}  // namespace

int orthogonalize(const OrthoCall& c, int dev, DeviceState& st, cudaStream_t s) {
    std::call_once(st.ortho_once, [&] { st.ortho_status = set_up_kernels(); });
    if (st.ortho_status != SGEMM_OK) return st.ortho_status;
    const int m = std::min(c.M, c.N);
    const long long pitch = (c.N + 15ll) / 16 * 16, mp = (m + 15ll) / 16 * 16;  // (the epilogue's accesses of 32 bytes)
    const int parts = c.type == SGEMM_TYPE_BF16 ? 1 : 2;
    // Row chunks of about 8192 elements, a few rounds of the GPU at most.
    OrthoPrep prep = {};
    prep.chunks = static_cast<int>(std::max(1ll, std::min({static_cast<long long>(kOrthoMostChunks), static_cast<long long>(c.M),
                                                           static_cast<long long>(c.M) * pitch / 8192})));
    prep.per = static_cast<int>(ceil_div(c.M, prep.chunks));
    prep.chunks = static_cast<int>(ceil_div(c.M, prep.per));
    if (static_cast<long long>(c.E) * prep.chunks > 0x7fffffffll) return SGEMM_ERR_INVALID_ARG;
    auto whole = [](long long bytes) { return (bytes + 255) / 256 * 256; };
    const long long xb = whole(2ll * 2 * c.E * c.M * pitch), ab = whole(2ll * 2 * c.E * m * mp);
    const long long db = whole(4ll * c.E * mp), pb = whole(8ll * c.E * prep.chunks);
    Workspace ws;
    ws.s = s;
    cudaMemPool_t pool = workspace_pool(dev, st);
    const long long bytes = (c.steps > 1 ? 2 : 1) * xb + 2 * ab + 2 * db + pb;
    if (!pool || cudaMallocFromPoolAsync(&ws.p, static_cast<size_t>(bytes), pool, s) != cudaSuccess) {
        (void)cudaGetLastError();
        ws.p = nullptr;
        return SGEMM_ERR_CUDA;
    }
    char* at = static_cast<char*>(ws.p);
    auto take = [&](long long n) {
        char* const q = at;
        at += n;
        return q;
    };
    prep.part = reinterpret_cast<double*>(take(pb));
    float* const d = reinterpret_cast<float*>(take(db));
    float* const e = reinterpret_cast<float*>(take(db));
    char* const a = take(ab);
    char* const b = take(ab);
    char* const x0 = take(xb);
    char* const x[2] = {x0, c.steps > 1 ? take(xb) : x0};
    prep.G = c.G, prep.ldg = c.ldg, prep.sg = c.sg;
    prep.E = c.E, prep.rows = c.M, prep.cols = c.N;
    prep.vec = row_alignment(c.G, c.type == SGEMM_TYPE_F32 ? 4 : 2, c.M > 1 ? c.ldg : 0, c.E > 1 ? c.sg : 0) == 16;
    prep.eps = c.eps;
    prep.hi = reinterpret_cast<uint16_t*>(x0), prep.pitch = pitch, prep.plane = static_cast<long long>(c.E) * c.M * pitch;
    const int rc = ortho_prepare(prep, c.type, s);
    if (rc != SGEMM_OK) return rc;
    // Pairs of CTAs where their tiles are half as many as the pairs at least, else
    // single CTAs with tiles of 128 x 128.
    const long long wide = parts == 1 ? 256 : 128;
    const long long tiles = c.E * ceil_div(c.M, wide) * ceil_div(c.N, 256);
    const bool pairs = 2 * tiles >= st.max_pairs;
    if (parts == 1)
        return pairs ? steps<256, 2, 1>(c, prep, x, a, b, d, e, st, s) : steps<128, 1, 1>(c, prep, x, a, b, d, e, st, s);
    return pairs ? steps<128, 2, 2>(c, prep, x, a, b, d, e, st, s) : steps<128, 1, 2>(c, prep, x, a, b, d, e, st, s);
}

}  // namespace detail
}  // namespace gb300
