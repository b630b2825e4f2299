// serving_api.cu -- the entry points of include/rmsnorm_serving.h: argument checks, launch
// shapes and launches of the kernels in matmul.cu, weight.cu and append.cu.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <map>
#include <mutex>
#include <utility>

#include "../../include/rmsnorm_serving.h"
#include "checks.h"
#include "fused.h"
#include "launch.h"
#include "serving.h"
#include "tuning.h"

namespace rmsnorm {
namespace {

constexpr int64_t kMatmulMost = RMSNORM_MATMUL_MAX;
constexpr int64_t kBlock = RMSNORM_MATMUL_BLOCK;

cudaLaunchConfig_t launch_config(int64_t blocks, int threads, size_t smem, int cluster, cudaStream_t s,
                                 cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

cudaError_t launch(const void* k, int64_t blocks, int threads, size_t smem, int cluster, void** params, cudaStream_t s) {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = launch_config(blocks, threads, smem, cluster, s, attr);
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, k, params);
}

// Launch, and once more after the kernel's attributes are set again, which a device reset
// since the first call discards.
rmsnorm_status run(const void* k, int64_t blocks, int threads, size_t smem, int cluster, void** params, rmsnorm_stream_t stream) {
    if (!k) return RMSNORM_ERR_UNSUPPORTED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return RMSNORM_ERR_CUDA;
    if (smem > 48 * 1024 && resident_blocks(k, dev, threads, smem) < 1) {
        (void)cudaGetLastError();
        return RMSNORM_ERR_CUDA;
    }
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (launch(k, blocks, threads, smem, cluster, params, s) == cudaSuccess) return RMSNORM_OK;
    (void)cudaGetLastError();
    if (smem > 48 * 1024 && allow_shared_memory(k, dev) && launch(k, blocks, threads, smem, cluster, params, s) == cudaSuccess)
        return RMSNORM_OK;
    (void)cudaGetLastError();
    return RMSNORM_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// tensor maps
// ---------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// Rows that TMA takes: on 16-byte boundaries (one row alone has no pitch).
bool tma_rows(const void* p, int64_t ld, int64_t rows) { return aligned(p, 16) && (rows <= 1 || ld % 16 == 0); }

// Boxes of `box` rows of 128 codes of a matrix [rows, K], swizzled by 128 bytes; what lies
// outside of it reads as zero.
bool tile_map(CUtensorMap& map, const void* p, int64_t ld, int64_t rows, int64_t K, int box) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(rows > 1 ? ld : round_up(K, 16))};
    const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(kBlock), static_cast<cuuint32_t>(box)};
    const cuuint32_t steps[2] = {1, 1};
    return encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, boxes, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of 1, 2, ... blocks that the device holds at a time.
struct ClusterFits {
    int of[kMatmulMostSplit + 1] = {};
};
std::mutex g_serving_mu;
std::map<std::pair<const void*, int>, ClusterFits> g_clusters;  // by (kernel, device)

// Those of the plan's blocks; false on failure. Fewer than the SMs would hold where their groups
// are no multiple of a cluster: 48 clusters of 6 blocks, two to an SM, do not fit 152 SMs.
bool cluster_fits(const MatmulPlan& p, int dev, ClusterFits& fits) {
    const void* k = matmul_kernel(p);
    if (!k) return false;
    try {
        {
            std::lock_guard<std::mutex> lock(g_serving_mu);
            const auto found = g_clusters.find({k, dev});
            if (found != g_clusters.end()) {
                fits = found->second;
                return true;
            }
        }
        if (resident_blocks(k, dev, p.threads, p.smem) < 1) return false;
        for (int n = 2; n <= kMatmulMostSplit; ++n) {
            cudaLaunchAttribute attr[1];
            const cudaLaunchConfig_t cfg = launch_config(n, p.threads, p.smem, n, nullptr, attr);
            if (cudaOccupancyMaxActiveClusters(&fits.of[n], k, &cfg) != cudaSuccess) return false;
        }
        std::lock_guard<std::mutex> lock(g_serving_mu);
        g_clusters[{k, dev}] = fits;
        return true;
    } catch (...) {
        return false;
    }
}

std::atomic<int> g_give_up{-1};  // rmsnorm_selftest_matmul_gives_up

// How a product is cut; false on failure. Few rows of a: b's rows in the accumulators' lanes.
// More: 128 x 128 by single blocks or 256 x 256 by pairs, whichever takes less, a turn of
// the pairs taking as long as 1.55 of the others' (N = K = 4096: 512 rows 12.6 us and 17.1,
// 1024 rows 22.4 and 18.2, 8192 rows 142 and 111). Where tiles leave half of the SMs without one, K is
// shared by as many blocks as the GPU holds at a time.
bool matmul_plan(int64_t M, int64_t N, int64_t K, bool tma, int dtype, int dev, int sms, MatmulPlan& p) {
    p.dtype = dtype;
    p.tma = tma;
    const int64_t wide = ceil_div(M, 128) * ceil_div(N, 128), pairs = ceil_div(M, 256) * ceil_div(N, 256);
    if (M <= 64) {
        p.how = kMatmulThin;
        for (p.n = 16; p.n < M;) p.n *= 2;
    } else {
        p.how = !tma || 100 * ceil_div(wide, sms) <= 155 * ceil_div(pairs, sms / 2) ? kMatmulWide : kMatmulPair;
    }
    matmul_shape(p);
    if (p.how == kMatmulPair) {
        p.cluster = 2;
        p.blocks = 2 * std::min<int64_t>(pairs, sms / 2);
        return true;
    }
    const int64_t tiles = p.how == kMatmulThin ? ceil_div(M, p.n) * ceil_div(N, 128) : wide;
    // (four blocks of K at least to each in tiles of 128 x 128, whose sums take longer to meet)
    const int64_t parts = p.how == kMatmulThin ? ceil_div(K, kBlock) : std::max<int64_t>(1, K / (4 * kBlock));
    p.cluster = static_cast<int>(std::min<int64_t>(kMatmulMostSplit, parts));
    if (p.cluster > 1) {
        ClusterFits fits;
        if (!cluster_fits(p, dev, fits)) return false;
        while (p.cluster > 1 && tiles > fits.of[p.cluster]) --p.cluster;
    }
    p.blocks = p.cluster > 1 || p.how == kMatmulThin ? tiles * p.cluster : std::min<int64_t>(tiles, sms);
    return true;
}

// Rows of a tile of a and of b, and of the boxes that are loaded.
int tile_rows_a(const MatmulPlan& p) { return p.how == kMatmulThin ? p.n : p.how == kMatmulPair ? 256 : 128; }
int tile_rows_b(const MatmulPlan& p) { return p.how == kMatmulPair ? 256 : 128; }
int box_rows_a(const MatmulPlan& p) { return p.how == kMatmulThin ? p.n : 128; }

// Whether [p, p + bytes) and [q, q + more) share memory.
bool overlap(const void* p, int64_t bytes, const void* q, int64_t more) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && bytes > 0 && more > 0 && a < b + static_cast<uintptr_t>(more) && b < a + static_cast<uintptr_t>(bytes);
}

int64_t span(int64_t rows, int64_t ld, int64_t width, int64_t bytes) { return rows > 0 ? ((rows - 1) * ld + width) * bytes : 0; }

// Dimensions of a tensor by count and stride, outside of `inner` elements: whether no two of
// its elements meet (each stride steps over all that lies inside of it), and the elements
// from its first to behind its last.
struct Dim {
    int64_t count, stride;
};
bool nested(std::initializer_list<Dim> dims, int64_t inner, int64_t& extent) {
    Dim d[4];
    int n = 0;
    for (const Dim& x : dims)
        if (x.count > 1) d[n++] = x;
    std::sort(d, d + n, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
    extent = inner;
    for (int i = 0; i < n; ++i) {
        if (d[i].stride < extent || d[i].stride > (int64_t(1) << 46) / d[i].count) return false;
        extent += (d[i].count - 1) * d[i].stride;
    }
    return extent <= int64_t(1) << 46;
}

// Whether two caches of one kind of rows keep out of each other: apart, or, of the same
// strides, interleaved as the halves of one tensor.
bool caches_apart(const void* p, const void* q, int64_t span_p, int64_t span_q, int64_t bytes, bool same, const Dim& page,
                  const Dim& row, const Dim& head, int64_t inner) {
    if (!overlap(p, span_p, q, span_q)) return true;
    const int64_t apart = reinterpret_cast<intptr_t>(q) - reinterpret_cast<intptr_t>(p);
    int64_t all;
    return same && apart % bytes == 0 && nested({page, row, head, {2, std::abs(apart / bytes)}}, inner, all);
}

bool dtype_ok(rmsnorm_dtype dt) { return dt == RMSNORM_F32 || dt == RMSNORM_F16 || dt == RMSNORM_BF16; }

}  // namespace
}  // namespace rmsnorm

using namespace rmsnorm;

extern "C" rmsnorm_status rmsnorm_quant_weight(const void* w, int64_t ldw, void* codes, int64_t ldcodes, float* scales,
                                               int64_t ldscales, int64_t N, int64_t K, rmsnorm_dtype dtype, int pow2,
                                               rmsnorm_stream_t stream) {
    if (!dtype_ok(dtype)) return RMSNORM_ERR_DTYPE;
    if (pow2 != 0 && pow2 != 1) return RMSNORM_ERR_ARG;
    const size_t s = elem_bytes(dtype);
    if (N < 0 || N > kMatmulMost || K < 1 || K > kMatmulMost) return RMSNORM_ERR_SHAPE;
    const int64_t kblocks = ceil_div(K, kBlock), nblocks = ceil_div(N, kBlock);
    if (!pitch_ok(ldw, K, N, s) || !pitch_ok(ldcodes, K, N, 1) || !pitch_ok(ldscales, kblocks, nblocks, 4))
        return RMSNORM_ERR_SHAPE;
    if (N == 0) return RMSNORM_OK;
    if (!w || !codes || !scales) return RMSNORM_ERR_NULL;
    if (!aligned(w, s) || !aligned(scales, 4)) return RMSNORM_ERR_ALIGN;
    const int64_t wb = span(N, ldw, K, s), cb = span(N, ldcodes, K, 1), sb = span(nblocks, ldscales, kblocks, 4);
    if (overlap(w, wb, codes, cb) || overlap(w, wb, scales, sb) || overlap(codes, cb, scales, sb)) return RMSNORM_ERR_ARG;
    WeightArgs a = {};
    a.w = w;
    a.codes = codes;
    a.scales = scales;
    a.ldw = ldw;
    a.ldcodes = ldcodes;
    a.ldscales = ldscales;
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.kblocks = static_cast<int>(kblocks);
    a.pow2 = pow2;
    const bool wide = K % 8 == 0 && aligned(w, 16) && ldw * static_cast<int64_t>(s) % 16 == 0 && aligned(codes, 8) &&
                      ldcodes % 8 == 0;
    void* params[] = {&a};
    return run(weight_kernel(dtype, wide), nblocks * kblocks, weight_threads(), 0, 1, params, stream);
}

extern "C" rmsnorm_status rmsnorm_quant_matmul(const void* a, int64_t lda, const float* a_scales, int64_t ldas, const void* b,
                                               int64_t ldb, const float* b_scales, int64_t ldbs, const void* bias, void* y,
                                               int64_t ldy, int64_t M, int64_t N, int64_t K, rmsnorm_dtype dtype, int group,
                                               rmsnorm_stream_t stream) {
    if (!dtype_ok(dtype)) return RMSNORM_ERR_DTYPE;
    if (group != 0 && group != kBlock) return RMSNORM_ERR_ARG;
    if (M < 0 || M > RMSNORM_MAX_M || N < 1 || N > kMatmulMost || K < 1 || K > kMatmulMost) return RMSNORM_ERR_SHAPE;
    const size_t s = elem_bytes(dtype);
    const int64_t kblocks = ceil_div(K, kBlock), nblocks = ceil_div(N, kBlock), per_row = group ? kblocks : 1;
    if (!pitch_ok(lda, K, M, 1) || !pitch_ok(ldas, per_row, M, 4) || !pitch_ok(ldb, K, N, 1) ||
        !pitch_ok(ldbs, kblocks, nblocks, 4) || !pitch_ok(ldy, N, M, s))
        return RMSNORM_ERR_SHAPE;
    if (M == 0) return RMSNORM_OK;
    if (!a || !a_scales || !b || !b_scales || !y) return RMSNORM_ERR_NULL;
    if (!aligned(a_scales, 4) || !aligned(b_scales, 4) || !aligned(bias, s) || !aligned(y, s)) return RMSNORM_ERR_ALIGN;
    const int64_t yb = span(M, ldy, N, s);
    if (overlap(y, yb, a, span(M, lda, K, 1)) || overlap(y, yb, a_scales, span(M, ldas, per_row, 4)) ||
        overlap(y, yb, b, span(N, ldb, K, 1)) || overlap(y, yb, b_scales, span(nblocks, ldbs, kblocks, 4)) ||
        overlap(y, yb, bias, N * s))
        return RMSNORM_ERR_ARG;
    int dev = 0;
    const int sms = current_sms(dev);
    if (!sms) {
        (void)cudaGetLastError();
        return RMSNORM_ERR_CUDA;
    }
    MatmulPlan p;
    if (!matmul_plan(M, N, K, tma_rows(a, lda, M) && tma_rows(b, ldb, N), dtype, dev, sms, p)) {
        (void)cudaGetLastError();
        return RMSNORM_ERR_CUDA;
    }
    MatmulArgs t = {};
    t.a = static_cast<const uint8_t*>(a);
    t.sa = a_scales;
    t.b = static_cast<const uint8_t*>(b);
    t.sb = b_scales;
    t.bias = bias;
    t.y = y;
    t.lda = lda;
    t.ldsa = ldas;
    t.ldb = ldb;
    t.ldsb = ldbs;
    t.ldy = ldy;
    t.M = M;
    t.N = static_cast<int>(N);
    t.K = static_cast<int>(K);
    t.kblocks = static_cast<int>(kblocks);
    t.per_row = group == 0;
    t.m_tiles = static_cast<int>(ceil_div(M, tile_rows_a(p)));
    t.n_tiles = static_cast<int>(ceil_div(N, tile_rows_b(p)));
    t.wide_y = aligned(y, 16) && ldy * static_cast<int64_t>(s) % 16 == 0;
    t.wide_bias = bias && aligned(bias, 16);
    t.give_up = g_give_up.load(std::memory_order_relaxed);
    t.err = device_error_word();
    if (!t.err) return RMSNORM_ERR_CUDA;
    CUtensorMap amap = {}, bmap = {};
    if (p.tma && (!tile_map(amap, a, lda, M, K, box_rows_a(p)) || !tile_map(bmap, b, ldb, N, K, 128)))
        return RMSNORM_ERR_CUDA;
    void* params[] = {&t, &amap, &bmap};
    return run(matmul_kernel(p), p.blocks, p.threads, p.smem, p.cluster, params, stream);
}

extern "C" rmsnorm_status rmsnorm_selftest_matmul_gives_up(int rank) {
#ifdef RMSNORM_DEBUG
    if (rank < -1 || rank >= kMatmulMostSplit) return RMSNORM_ERR_ARG;
    g_give_up.store(rank, std::memory_order_relaxed);
    return RMSNORM_OK;
#else
    (void)rank;
    return RMSNORM_ERR_UNSUPPORTED;
#endif
}

extern "C" rmsnorm_status rmsnorm_rope_append(const rmsnorm_rope_heads* q, const rmsnorm_cache_heads* k,
                                              const rmsnorm_cache_heads* v, const int64_t* slots, int64_t pages,
                                              int64_t page_size, const int64_t* positions, int64_t T, int64_t D,
                                              int64_t rotary_dim, const double* inv_freq, int interleaved, float mscale,
                                              float eps, rmsnorm_dtype dtype, int offset, rmsnorm_stream_t stream) {
    rmsnorm_status st = check_rope(1, T, D, rotary_dim, interleaved, mscale, eps, dtype, offset);
    if (st != RMSNORM_OK) return st;
    if (!k) return RMSNORM_ERR_NULL;
    if (pages < 1 || page_size < 1 || page_size > INT32_MAX || pages > (int64_t(1) << 46) / page_size) return RMSNORM_ERR_SHAPE;
    const int64_t s = elem_bytes(dtype);
    AppendArgs a = {};
    bool wide = true, codes = false;
    int64_t heads = 0, bytes[3] = {0, 0, 0}, extent[3] = {0, 0, 0}, scale_extent[3] = {0, 0, 0};
    if (q) {
        if (q->heads < 1 || q->heads > RMSNORM_ROPE_MAX_HEADS || !strides_ok(q->x_token, q->x_head, q->heads, T, D) ||
            !output_strides_ok(q->y_token, q->y_head, q->heads, T, D))
            return RMSNORM_ERR_SHAPE;
        AppendSet& t = a.sets[0];
        t.x = q->x;
        t.gamma = q->gamma;
        t.y = q->y;
        t.x_token = q->x_token;
        t.x_head = q->x_head;
        t.y_token = q->y_token;
        t.y_head = q->y_head;
        t.heads = static_cast<int>(q->heads);
        bytes[0] = s;
        extent[0] = T > 0 ? (T - 1) * q->y_token + (q->heads - 1) * q->y_head + D : 0;
        heads += q->heads;
    }
    for (int i = 1; i < 3; ++i) {
        const rmsnorm_cache_heads* c = i == 1 ? k : v;
        if (!c) continue;
        if (c->heads < 1 || c->heads > RMSNORM_ROPE_MAX_HEADS || !strides_ok(c->x_token, c->x_head, c->heads, T, D) ||
            !nested({{pages, c->page}, {page_size, c->row}, {c->heads, c->head}}, D, extent[i]) ||
            (c->scales &&
             !nested({{pages, c->scale_page}, {page_size, c->scale_row}, {c->heads, c->scale_head}}, 1, scale_extent[i])))
            return RMSNORM_ERR_SHAPE;
        if (i == 2 && c->gamma) return RMSNORM_ERR_ARG;  // values are not normalised
        AppendSet& t = a.sets[i];
        t.x = c->x;
        t.gamma = c->gamma;
        t.y = c->rows;
        t.x_token = c->x_token;
        t.x_head = c->x_head;
        t.y_page = c->page;
        t.y_token = c->row;
        t.y_head = c->head;
        t.scales = c->scales;
        t.scale_page = c->scale_page;
        t.scale_row = c->scale_row;
        t.scale_head = c->scale_head;
        t.heads = static_cast<int>(c->heads);
        bytes[i] = c->scales ? 1 : s;
        codes = codes || c->scales;
        heads += c->heads;
    }
    if (heads > RMSNORM_ROPE_MAX_HEADS) return RMSNORM_ERR_SHAPE;
    if (T == 0) return RMSNORM_OK;
    const int64_t words = 16 / s;
    for (int i = 0; i < 3; ++i) {
        const AppendSet& t = a.sets[i];
        if (!t.heads) continue;
        if (!t.x || !t.y) return RMSNORM_ERR_NULL;
        if (!aligned(t.x, s) || !aligned(t.gamma, s) || !aligned(t.y, bytes[i]) || !aligned(t.scales, 4)) return RMSNORM_ERR_ALIGN;
        const int64_t w = t.scales ? 8 : words;
        wide = wide && aligned(t.x, 16) && aligned(t.gamma, 16) && t.x_token % words == 0 && t.x_head % words == 0 &&
               aligned(t.y, t.scales ? 8 : 16) && t.y_page % w == 0 && t.y_token % w == 0 && t.y_head % w == 0;
    }
    // the queries' output may be the queries, or lie between other heads of their rows
    if (q) {
        const HeadsAt out = {q->y, q->y_token, q->y_head, q->heads};
        for (int j = 0; j < 3; ++j) {
            const AppendSet& t = a.sets[j];
            const HeadsAt in = {t.x, t.x_token, t.x_head, t.heads};
            if (t.heads && !(j == 0 && heads_same(out, in, T)) && !heads_apart(out, in, T, D, s)) return RMSNORM_ERR_ARG;
        }
    }
    if (!slots || !positions || !inv_freq) return RMSNORM_ERR_NULL;
    if (!aligned(slots, 8) || !aligned(positions, 8) || !aligned(inv_freq, 8)) return RMSNORM_ERR_ALIGN;
    // what else is written against what is read and written
    for (int i = 0; i < 3; ++i) {
        const AppendSet& o = a.sets[i];
        if (!o.heads) continue;
        for (int j = 0; j < 3; ++j) {
            const AppendSet& t = a.sets[j];
            if (!t.heads) continue;
            const int64_t read = ((T - 1) * t.x_token + (t.heads - 1) * t.x_head + D) * s;
            if (i > 0 && overlap(o.y, extent[i] * bytes[i], t.x, read)) return RMSNORM_ERR_ARG;
            if (overlap(o.y, extent[i] * bytes[i], t.gamma, D * s) || overlap(o.scales, scale_extent[i] * 4, t.x, read) ||
                overlap(o.scales, scale_extent[i] * 4, t.gamma, D * s) ||
                overlap(o.scales, scale_extent[i] * 4, t.y, extent[j] * bytes[j]))
                return RMSNORM_ERR_ARG;
        }
        if (i > 0 && overlap(o.y, extent[i] * bytes[i], a.sets[0].y, extent[0] * bytes[0])) return RMSNORM_ERR_ARG;
        for (const void* p : {static_cast<const void*>(slots), static_cast<const void*>(positions)})
            if (overlap(o.y, extent[i] * bytes[i], p, T * 8) || overlap(o.scales, scale_extent[i] * 4, p, T * 8))
                return RMSNORM_ERR_ARG;
        if (overlap(o.y, extent[i] * bytes[i], inv_freq, rotary_dim * 4) ||
            overlap(o.scales, scale_extent[i] * 4, inv_freq, rotary_dim * 4))
            return RMSNORM_ERR_ARG;
    }
    if (v) {
        const AppendSet &x = a.sets[1], &y = a.sets[2];
        const int most = std::max(x.heads, y.heads);
        const bool same = bytes[1] == bytes[2] && x.y_page == y.y_page && x.y_token == y.y_token && x.y_head == y.y_head;
        if (!caches_apart(x.y, y.y, extent[1] * bytes[1], extent[2] * bytes[2], bytes[1], same, {pages, x.y_page},
                          {page_size, x.y_token}, {most, x.y_head}, D))
            return RMSNORM_ERR_ARG;
        const bool same_scales = x.scale_page == y.scale_page && x.scale_row == y.scale_row && x.scale_head == y.scale_head;
        if (x.scales && y.scales &&
            !caches_apart(x.scales, y.scales, scale_extent[1] * 4, scale_extent[2] * 4, 4, same_scales, {pages, x.scale_page},
                          {page_size, x.scale_row}, {most, x.scale_head}, 1))
            return RMSNORM_ERR_ARG;
    }
    int dev = 0;
    const int sms = current_sms(dev);
    if (!sms) {
        (void)cudaGetLastError();
        return RMSNORM_ERR_CUDA;
    }
    a.heads = static_cast<int>(heads);
    a.pos = positions;
    a.inv_freq = inv_freq;
    a.T = T;
    a.D = static_cast<int>(D);
    a.R = static_cast<int>(rotary_dim);
    a.interleaved = interleaved;
    a.mscale = mscale;
    a.eps = eps;
    a.one = static_cast<float>(offset);
    a.slots = slots;
    a.pages = pages;
    a.page_size = static_cast<int>(page_size);
    a.err = device_error_word();
    if (!a.err) return RMSNORM_ERR_CUDA;
    RopePlan p;
    p.dtype = dtype;
    rope_lanes(D, rotary_dim, interleaved, wide, p);
    // heads to a group as in the rotation alone (rope_plan): a batch where the tokens fill the GPU,
    // fewer where they do not; and a run of heads where a group's turns take longer (bf16
    // 8192 x 48 x 90 110 us with 8 heads, 116 with 4, 120 with 16)
    const int64_t full = static_cast<int64_t>(sms) * (p.rows == kRopeSwap ? 512 : 1024) / p.lanes;
    const int64_t most = p.rows == kRopeEntries || p.rows == kRopeSwap ? kRopeRun : rope_fwd_batch(dtype);
    a.chunk = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, T * heads / full)));
    p.blocks = 0;
    for (int i = 0; i < 3; ++i) {
        a.first[i] = static_cast<int>(std::min<int64_t>(p.blocks, INT32_MAX));
        p.blocks += ceil_div(T * ceil_div(a.sets[i].heads, a.chunk), p.threads / p.lanes);
    }
    if (p.blocks > INT32_MAX) return RMSNORM_ERR_SHAPE;
    void* params[] = {&a};
    return run(append_kernel(p, codes), p.blocks, p.threads, 0, 1, params, stream);
}
