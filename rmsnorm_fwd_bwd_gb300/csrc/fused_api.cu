// fused_api.cu -- the entry points of include/rmsnorm_fused.h: argument checks,
// launch shapes and launches of the kernels in add.cu, quant.cu and rope.cu.
#include <algorithm>
#include <cmath>
#include <map>
#include <mutex>
#include <numeric>
#include <utility>

#include "../../include/rmsnorm_fused.h"
#include "checks.h"
#include "fused.h"
#include "launch.h"

namespace rmsnorm {
namespace {

static_assert(kRopeMaxSets == RMSNORM_ROPE_MAX_SETS, "sets of a rope call");

// Fewest rows that the backward's ring takes: fewer do not fill it (bf16 1023 x 4096
// 16.9 us without it, 1024 x 4096 15.7 with it).
constexpr int64_t kRingLeastRows = 1024;

// The rotation's backward's blocks per SM (what its registers leave).
constexpr int kRopeBwdBlocks = 3;

std::mutex g_fused_mu;
std::map<int, int> g_fused_sms;                                   // SMs by device
std::map<std::pair<const void*, std::pair<int, int>>, int> g_fused_fit;  // resident blocks per SM by (kernel, (device, threads))

}  // namespace

// SMs of the current device; 0 on failure.
int current_sms(int& dev) {
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    try {
        std::lock_guard<std::mutex> lock(g_fused_mu);
        int& n = g_fused_sms[dev];
        if (n == 0 && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) n = 0;
        return n;
    } catch (...) {  // no memory for the entry: nothing is thrown through the C entry points
        return 0;
    }
}

// Allow the kernel the device's whole shared memory; the attribute belongs to the
// context, so it is set again where a launch fails (run).
bool allow_shared_memory(const void* k, int dev) {
    int optin = 0;
    cudaFuncAttributes fa;
    return cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) == cudaSuccess &&
           cudaFuncGetAttributes(&fa, k) == cudaSuccess &&
           cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, optin - static_cast<int>(fa.sharedSizeBytes)) ==
               cudaSuccess &&
           cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) ==
               cudaSuccess;
}

// Blocks of `threads` that an SM holds, for the persistent kernels; 0 on failure.
int resident_blocks(const void* k, int dev, int threads, size_t smem) {
    try {
        std::lock_guard<std::mutex> lock(g_fused_mu);
        int& n = g_fused_fit[{k, {dev, static_cast<int>(smem) * 1024 + threads}}];
        if (n == 0 && ((smem > 48 * 1024 && !allow_shared_memory(k, dev)) ||
                       cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k, threads, smem) != cudaSuccess))
            n = 0;
        return n;
    } catch (...) {
        return 0;
    }
}

namespace {

cudaError_t launch(const void* k, int64_t blocks, int threads, size_t smem, void** params, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, k, params);
}

// Octets of a row that may start off a 16-byte boundary (`wide`: it does not).
int64_t octets_of(int64_t N, int dtype, bool wide) { return wide ? N / 8 : ceil_div(N + (dtype == RMSNORM_F32 ? 3 : 7), 8); }

// The fewest threads, a multiple of 32, that hold n octets, times their octets, over
// the given choices of octets per thread; the first of equals.
bool block_shape(int64_t n, std::initializer_list<int> choices, int most, AddPlan& p) {
    int64_t best = 0;
    for (const int octets : choices) {
        const int64_t threads = round_up(ceil_div(n, octets), 32);
        if (threads > most || (best && threads * octets >= best)) continue;
        best = threads * octets;
        p.octets = octets;
        p.threads = static_cast<int>(threads);
    }
    return best > 0;
}

// Lanes per row and octets per thread for rows of n octets: up to 128 (64 off 16 bytes,
// where a row's ends cost a warp more) by groups of lanes of a 4-warp block (the 8-bit
// output wants a warp, whose neighbouring lanes hold a group of columns), wider rows by
// a block.
bool row_shape(int64_t n, int least_lanes, std::initializer_list<int> choices, AddPlan& p) {
    // (65536 x 513 bf16 off 16 bytes 166 us by lanes, 147 by blocks; 65536 x 1000 with an 8-bit
    // output 66 by lanes, 70 by blocks)
    if (n <= (p.mode == kRowsOnePhase ? 64 : 128)) {
        p.lanes = n <= 16 ? least_lanes : 32;
        p.octets = 1;
        while (static_cast<int64_t>(p.lanes) * p.octets < n) p.octets *= 2;
        p.threads = kFusedGroupThreads;
        return true;
    }
    p.lanes = 0;
    return block_shape(n, choices, kFusedMaxThreads, p);
}

// The forwards' shape: four octets a thread of aligned rows (two with as few threads
// idle); two of others, whose shifting and masking hold registers, in wide blocks where
// kFusedMaxThreads do not hold the row. bf16 with dropout: 16384 x 4096 78.9 us with four,
// 84.4 with two; 16384 x 14278 667 us with three octets of 608 threads, 533 in wide blocks.
bool fwd_shape(int64_t n, int least_lanes, AddPlan& p) {
    if (p.mode == kRowsAligned) return row_shape(n, least_lanes, {4, 2}, p);
    if (row_shape(n, least_lanes, {2}, p)) return true;
    p.lanes = -1;
    return block_shape(n, {2, 3}, kFusedWideThreads, p);
}

int64_t rows_per_block(const AddPlan& p) { return p.lanes > 0 ? p.threads / p.lanes : 1; }

struct Operand {
    const void* p;
    int64_t ld;
};

// Whether the rows of all operands start at one offset from a 16-byte boundary, row by
// row.
bool one_offset(size_t s, std::initializer_list<Operand> operands) {
    const Operand* q = nullptr;
    for (const Operand& o : operands) {
        if (!o.p) continue;
        if (q && (((reinterpret_cast<uintptr_t>(o.p) ^ reinterpret_cast<uintptr_t>(q->p)) & 15) != 0 ||
                  (o.ld - q->ld) * static_cast<int64_t>(s) % 16 != 0))
            return false;
        q = &o;
    }
    return true;
}

// No two of the given outputs (NULL: not written) at one address.
bool distinct(std::initializer_list<const void*> outputs) {
    for (auto p = outputs.begin(); p != outputs.end(); ++p)
        for (auto q = outputs.begin(); *p && q != p; ++q)
            if (*p == *q) return false;
    return true;
}

// Whether the output's rows (NULL: not written) are those of each input at its address: of
// one pitch (the weight has pitch 0: all rows read it).
bool same_rows(int64_t M, const Operand& out, std::initializer_list<Operand> inputs) {
    for (const Operand& in : inputs)
        if (out.p && out.p == in.p && M > 1 && out.ld != in.ld) return false;
    return true;
}

RowMode row_mode(bool wide, bool one) { return wide ? kRowsAligned : one ? kRowsOnePhase : kRowsAny; }

// Every row of every operand on a 16-byte boundary (8 for 1-byte elements), and
// whole octets.
bool wide_rows(int64_t N, size_t s, std::initializer_list<Operand> operands) {
    if (N % 8 != 0) return false;
    for (const Operand& o : operands)
        if (o.p && (!aligned(o.p, s == 1 ? 8 : 16) || (o.ld * static_cast<int64_t>(s)) % (s == 1 ? 8 : 16) != 0)) return false;
    return true;
}

bool check_dropout(float p, const uint64_t* rng, AddArgs& a, rmsnorm_status& st) {
    if (!(p >= 0.0f && p <= 1.0f)) {
        st = RMSNORM_ERR_ARG;
        return false;
    }
    a.threshold = static_cast<uint32_t>(std::lround(65536.0 * static_cast<double>(p)));
    a.scale = a.threshold < 65536u ? static_cast<float>(65536.0 / (65536 - static_cast<int>(a.threshold))) : 0.0f;
    a.rng = reinterpret_cast<const unsigned long long*>(rng);
    return true;
}

rmsnorm_status check_rng(const AddArgs& a) {
    if (a.threshold && !a.rng) return RMSNORM_ERR_NULL;
    if (a.threshold && (!aligned(a.rng, 8) || !aligned(a.rng_used, 8))) return RMSNORM_ERR_ALIGN;
    return RMSNORM_OK;
}

// The ring's shape; false where it does not apply.
bool ring_plan(int64_t M, int64_t N, int dtype, RowMode mode, bool drop, bool has_dh, int dev, int sms, AddPlan& p) {
    // narrow aligned rows do as well by lanes (65536 x 1000 bf16 89 us either way), narrow ones
    // off 16 bytes do not (65536 x 1001 233 us by lanes, 104 by the ring)
    if (N <= (mode == kRowsAligned ? 1024 : 256) || M < kRingLeastRows) return false;
    const bool wide = mode == kRowsAligned;
    p.dtype = dtype;
    p.mode = mode;
    p.drop = drop;
    p.ring = true;
    const int64_t eb = elem_bytes(dtype);
    if (!block_shape(octets_of(N, dtype, wide), {2, 3, 4}, kFusedMaxThreads, p)) return false;
    // whole octets for every thread that has one: rows off 16 bytes are copied from the
    // word they start in to the one they end in
    const int64_t octet = 8 * eb;
    p.slot = static_cast<uint32_t>(wide ? N * eb : octets_of(N, dtype, wide) * octet);
    const int64_t stage = (has_dh ? 3 : 2) * static_cast<int64_t>(p.slot);
    const int64_t fixed = p.threads * p.octets * (p.octets == 2 ? 32 : octet) + 64 * 4;
    const int64_t room = 227 * 1024;
    const void* k = add_bwd_kernel(p);
    const int by_registers = k ? resident_blocks(k, dev, p.threads, 1024) : 0;
    if (by_registers < 1) return false;
    // three stages, and blocks of 512 threads an SM together; of 768 with dropout, whose
    // numbers take as many instructions as the rest, and for rows off 16 bytes (then of two
    // stages, where three do not fit). bf16 16384 x 4096: 91 us with 512, 95 with 768; with
    // dropout 65536 x 4096: 451 and 423 us
    int bps = std::min(by_registers, static_cast<int>(ceil_div(drop || !wide ? 768 : 512, p.threads)));
    int64_t stages = 3;
    while (stages > 2 && bps * (stages * (stage + 8) + fixed + 1024) > room) --stages;
    while (bps > 1 && bps * (stages * (stage + 8) + fixed + 1024) > room) --bps;
    if (stages * (stage + 8) + fixed > room) return false;
    p.stages = static_cast<int>(stages);
    p.smem = static_cast<size_t>(stages * (stage + 8) + fixed);
    const int fit = resident_blocks(k, dev, p.threads, p.smem);
    if (fit < 1) return false;
    p.blocks = std::min<int64_t>(static_cast<int64_t>(std::min(fit, bps)) * sms, M);
    // two rows a block at least, where the column reduce is as long as the rows (bf16 4000 x 500
    // 12.2 us, 14.5 with one, 13.0 with four; 1024 x 1001 9.3, 11.0, 10.2)
    p.blocks = std::min<int64_t>(p.blocks, std::max<int64_t>(sms, ceil_div(M, 2)));
    if (!wide) p.blocks = std::min<int64_t>(p.blocks / 8 * 8, round_up(M, 8));
    return true;
}

// Persistent grid of the backward and its partial rows. Rows off 16 bytes want a grid
// that is a multiple of 8; blocks without a row write a row of zeros.
bool add_bwd_plan(int64_t M, int64_t N, int dtype, RowMode mode, bool drop, bool has_dh, AddPlan& p) {
    int dev = 0;
    const int sms = current_sms(dev);
    if (!sms) return false;
    if (mode != kRowsAny && ring_plan(M, N, dtype, mode, drop, has_dh, dev, sms, p)) return true;
    p = AddPlan();
    const bool wide = mode == kRowsAligned;
    p.dtype = dtype;
    p.mode = mode;
    if (!(wide ? row_shape(octets_of(N, dtype, wide), 8, {2, 4}, p)
              : row_shape(octets_of(N, dtype, wide), 8, {2, 4, 5}, p)))
        return false;
    p.smem = p.lanes ? static_cast<size_t>(rows_per_block(p)) * N * 4 : 0;
    const void* k = add_bwd_kernel(p);
    const int fit = k ? resident_blocks(k, dev, p.threads, p.smem) : 0;
    if (fit < 1) return false;
    const int64_t most = static_cast<int64_t>(std::min(fit, 8)) * sms, need = ceil_div(M, rows_per_block(p));
    p.blocks = wide ? std::min(most, need) : std::min(most / 8 * 8, round_up(need, 8));
    return true;
}

rmsnorm_status run(const void* k, const AddPlan& p, AddArgs& a, rmsnorm_stream_t stream) {
    if (!k) return RMSNORM_ERR_UNSUPPORTED;
    if (p.ring) {
        a.stages = p.stages;
        a.slot = p.slot;
        a.err = device_error_word();
        if (!a.err) return RMSNORM_ERR_CUDA;
    }
    void* params[] = {&a};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (launch(k, p.blocks, p.threads, p.smem, params, s) == cudaSuccess) return RMSNORM_OK;
    (void)cudaGetLastError();
    // a device reset since the attribute was set discards it
    int dev = 0;
    if (p.smem > 48 * 1024 && cudaGetDevice(&dev) == cudaSuccess && allow_shared_memory(k, dev) &&
        launch(k, p.blocks, p.threads, p.smem, params, s) == cudaSuccess)
        return RMSNORM_OK;
    (void)cudaGetLastError();
    return RMSNORM_ERR_CUDA;
}

}  // namespace

// ---------------------------------------------------------------------------
// rope
// ---------------------------------------------------------------------------
bool strides_ok(int64_t token, int64_t head, int64_t heads, int64_t T, int64_t D) {
    if ((T > 1 && token < D) || (heads > 1 && head < D) || token < 0 || head < 0) return false;
    const int64_t most = int64_t(1) << 40;
    return (T <= 1 || token <= most / (T - 1)) && (heads <= 1 || head <= most / (heads - 1));
}

// Output rows must not overlap: tokens outside heads, or heads outside tokens.
bool output_strides_ok(int64_t token, int64_t head, int64_t heads, int64_t T, int64_t D) {
    return strides_ok(token, head, heads, T, D) &&
           (T <= 1 || heads <= 1 || token >= (heads - 1) * head + D || head >= (T - 1) * token + D);
}

namespace {

// n pieces of `bytes`, `step` bytes apart.
struct Pieces {
    int64_t n, step, bytes;
    int64_t extent() const { return (n - 1) * step + bytes; }
    int64_t period() const { return n > 1 ? step : 0; }
};

// Whether two pieces never meet, the second `d` bytes behind the first, when both recur every g bytes.
bool recurring_apart(int64_t p, int64_t q, int64_t d, int64_t g) {
    const int64_t r = (d % g + g) % g;
    return r >= p && r + q <= g;
}

bool pieces_apart(const Pieces& p, const Pieces& q, int64_t d) {
    if (d >= p.extent() || d + q.extent() <= 0) return true;
    const int64_t g = std::gcd(p.period(), q.period());
    return g > 0 && recurring_apart(p.bytes, q.bytes, d, g);
}

// The same of rows of pieces, np of them p_step apart and nq q_step apart. Where a row is no longer than the
// steps' common divisor g, a row of p can meet two rows of q alone: those at d modulo g and g before.
bool rows_apart(int64_t np, int64_t p_step, const Pieces& p, int64_t nq, int64_t q_step, const Pieces& q, int64_t d) {
    const int64_t g = std::gcd(np > 1 ? p_step : 0, nq > 1 ? q_step : 0);
    if (g == 0) return pieces_apart(p, q, d);
    if (p.extent() > g || q.extent() > g) return false;
    const int64_t r = (d % g + g) % g;
    return pieces_apart(p, q, r) && pieces_apart(p, q, r - g);
}

}  // namespace

bool heads_apart(const HeadsAt& p, const HeadsAt& q, int64_t T, int64_t D, int64_t s) {
    const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(q.p) - reinterpret_cast<uintptr_t>(p.p));
    // (the stride of a single token or head may be any number)
    const auto pieces = [&](int64_t n, int64_t stride) { return Pieces{n, n > 1 ? stride * s : 0, D * s}; };
    const Pieces pt = pieces(T, p.token), ph = pieces(p.heads, p.head), qt = pieces(T, q.token), qh = pieces(q.heads, q.head);
    if (d >= pt.extent() + ph.extent() - D * s || d + qt.extent() + qh.extent() - D * s <= 0) return true;
    // heads within tokens, tokens within heads, or both at once
    if (rows_apart(T, pt.step, ph, T, qt.step, qh, d) || rows_apart(p.heads, ph.step, pt, q.heads, qh.step, qt, d)) return true;
    const int64_t g = std::gcd(std::gcd(pt.period(), ph.period()), std::gcd(qt.period(), qh.period()));
    return g > 0 && recurring_apart(D * s, D * s, d, g);
}

bool heads_same(const HeadsAt& p, const HeadsAt& q, int64_t T) {
    return p.p == q.p && p.heads == q.heads && (T <= 1 || p.token == q.token) && (p.heads <= 1 || p.head == q.head);
}

rmsnorm_status check_rope(int nsets, int64_t T, int64_t D, int64_t R, int interleaved, float mscale, float eps,
                          rmsnorm_dtype dtype, int offset) {
    const rmsnorm_status st = check_common(T, D, dtype, offset);
    if (st != RMSNORM_OK) return st;
    if (D > RMSNORM_ROPE_MAX_D || R < 2 || R > D || R % 2 != 0) return RMSNORM_ERR_SHAPE;
    if (!std::isfinite(eps) || !(eps > 0.0f)) return RMSNORM_ERR_EPS;
    if (nsets < 1 || nsets > RMSNORM_ROPE_MAX_SETS || (interleaved != 0 && interleaved != 1) || !std::isfinite(mscale))
        return RMSNORM_ERR_ARG;
    return RMSNORM_OK;
}

void rope_lanes(int64_t D, int64_t R, int interleaved, bool wide, RopePlan& p) {
    if (wide && D % 8 == 0) p.rows = interleaved ? kRopeNeighbours : R % 16 == 0 ? kRopeHalves : kRopeSwap;
    p.threads = kFusedGroupThreads;
    if (p.rows != kRopeEntries) {
        const int64_t units = p.rows == kRopeHalves ? R / 16 + ceil_div(D - R, 16) : ceil_div(D, 16);
        for (p.lanes = 4; p.lanes < units;) p.lanes *= 2;
    } else {
        // up to four pairs a lane (eight of 32 lanes) and few lanes, whose sums take fewer steps
        const int64_t pairs = R / 2 + ceil_div(D - R, 2);
        for (p.lanes = 8; p.lanes < 32 && 4 * p.lanes < pairs;) p.lanes *= 2;
        p.pairs = static_cast<int>(ceil_div(pairs, p.lanes));
    }
}

namespace {

// Whether a set's output, where it meets an input of a set, is that set's heads, of the same
// strides (or its weight, of one row), and whether it keeps out of the other set's output.
bool outputs_ok(const RopeArgs& a, int64_t T, int64_t D, int64_t bytes, int nsets) {
    for (int i = 0; i < nsets; ++i) {
        const RopeSet& o = a.set[i];
        const HeadsAt out = {o.y, o.y_token, o.y_head, o.heads};
        for (int j = 0; j < nsets; ++j) {
            const RopeSet& s = a.set[j];
            const HeadsAt x = {s.x, s.x_token, s.x_head, s.heads}, dy = {s.dy, s.dy_token, s.dy_head, s.heads};
            const HeadsAt gamma = {s.gamma, 0, 0, 1}, other = {s.y, s.y_token, s.y_head, s.heads};
            for (const HeadsAt* in : {&x, &dy, &gamma})
                if (in->p && !(i == j && heads_same(out, *in, T)) && !heads_apart(out, *in, T, D, bytes)) return false;
            if (i < j && !heads_apart(out, other, T, D, bytes)) return false;
        }
    }
    return true;
}

bool rope_wide(const RopeSet& s, size_t e) {
    const int64_t w = 16 / static_cast<int64_t>(e);
    return aligned(s.x, 16) && aligned(s.gamma, 16) && aligned(s.dy, 16) && aligned(s.y, 16) && s.x_token % w == 0 &&
           s.x_head % w == 0 && s.dy_token % w == 0 && s.dy_head % w == 0 && s.y_token % w == 0 && s.y_head % w == 0;
}

// Lanes per head row, and the heads of a token that a group of lanes takes: all of
// them where the tokens alone fill the GPU (a token's cosines and sines are then
// computed once), fewer where they do not.
rmsnorm_status rope_plan(RopeArgs& a, int dtype, int interleaved, bool wide, bool bwd, RopePlan& p) {
    int dev = 0;
    const int sms = current_sms(dev);
    if (!sms) return RMSNORM_ERR_CUDA;
    p.dtype = dtype;
    rope_lanes(a.D, a.R, interleaved, wide, p);
    const int group = p.lanes;  // lanes that share an item
    // groups that fill the GPU: 1024 threads an SM, of which the registers leave 640 in the
    // forward and 384 in the backward (bf16 1024 x 40 x 128: forward 5.9 us, 8.8 by 2048
    // threads; backward 14.5, 19.4 by 2048, 15.9 by 640), or 512 where a token's turns take
    // longer (1536 x 40 x 128, 24 rotated: 9.7 us, 20.1 by 2048)
    const int64_t full = static_cast<int64_t>(sms) * (p.rows == kRopeSwap ? 512 : 1024) / group;
    p.smem = bwd ? static_cast<size_t>(p.threads / group) * a.D * 4 : 0;
    if (p.rows != kRopeEntries) {
        const int batch = bwd || p.rows == kRopeSwap ? kRopeRun : rope_fwd_batch(dtype);
        a.chunk = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(batch, a.T * a.heads / full)));
        a.chunks0 = static_cast<int>(ceil_div(a.set[0].heads, a.chunk));
        a.nchunk = a.chunks0 + static_cast<int>(a.nsets > 1 ? ceil_div(a.set[1].heads, a.chunk) : 0);
        p.blocks = ceil_div(a.T * a.nchunk, p.threads / group);
        if (bwd) p.blocks = std::min<int64_t>(p.blocks, static_cast<int64_t>(sms) * kRopeBwdBlocks);
        if (p.blocks > INT32_MAX) return RMSNORM_ERR_SHAPE;
    } else {
        const int64_t nchunk = std::min<int64_t>(ceil_div(full, a.T), a.heads);
        a.chunk = static_cast<int>(ceil_div(a.heads, nchunk));
        a.nchunk = static_cast<int>(ceil_div(a.heads, a.chunk));
        p.blocks = std::min<int64_t>(ceil_div(a.T * a.nchunk, p.threads / group), static_cast<int64_t>(sms) * (bwd ? 8 : 64));
    }
    a.units = p.blocks;
    a.ldws = workspace_pitch(a.D);
    return RMSNORM_OK;
}

rmsnorm_status rope_run(RopeArgs& a, const RopePlan& p, int interleaved, bool bwd, cudaStream_t s) {
    const void* k = rope_kernel(p, bwd);
    if (!k) return RMSNORM_ERR_UNSUPPORTED;
    a.interleaved = interleaved;
    void* params[] = {&a};
    if (launch(k, p.blocks, p.threads, p.smem, params, s) != cudaSuccess) {
        (void)cudaGetLastError();
        return RMSNORM_ERR_CUDA;
    }
    return RMSNORM_OK;
}

}  // namespace
}  // namespace rmsnorm

using namespace rmsnorm;

extern "C" rmsnorm_status rmsnorm_add_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldres,
                                          const void* gamma, void* h, int64_t ldh, void* y, int64_t ldy, float* rstd,
                                          int64_t M, int64_t N, float eps, rmsnorm_dtype dtype, int offset,
                                          float dropout_p, const uint64_t* rng, uint64_t* rng_used,
                                          rmsnorm_stream_t stream) {
    rmsnorm_status st = check_common(M, N, dtype, offset);
    if (st != RMSNORM_OK) return st;
    if (!std::isfinite(eps) || !(eps > 0.0f)) return RMSNORM_ERR_EPS;
    const size_t s = elem_bytes(dtype);
    if (!pitch_ok(ldx, N, M, s) || !pitch_ok(ldy, N, M, s) || (residual && !pitch_ok(ldres, N, M, s)) ||
        (h && !pitch_ok(ldh, N, M, s)))
        return RMSNORM_ERR_SHAPE;
    AddArgs a = {};
    if (!check_dropout(dropout_p, rng, a, st)) return st;
    if (M == 0) return RMSNORM_OK;
    if (!x || !gamma || !y) return RMSNORM_ERR_NULL;
    if (!distinct({h, y, rstd}) || !same_rows(M, {h, ldh}, {{x, ldx}, {residual, ldres}, {gamma, 0}}) ||
        !same_rows(M, {y, ldy}, {{x, ldx}, {residual, ldres}, {gamma, 0}}))
        return RMSNORM_ERR_ARG;
    if (!aligned(x, s) || !aligned(residual, s) || !aligned(gamma, s) || !aligned(h, s) || !aligned(y, s) ||
        !aligned(rstd, 4))
        return RMSNORM_ERR_ALIGN;
    a.rng_used = reinterpret_cast<unsigned long long*>(rng_used);
    if ((st = check_rng(a)) != RMSNORM_OK) return st;
    a.x = x;
    a.res = residual;
    a.gamma = gamma;
    a.h = h;
    a.y = y;
    a.rstd = rstd;
    a.ldx = ldx;
    a.ldres = ldres;
    a.ldh = ldh;
    a.ldy = ldy;
    a.M = M;
    a.N = static_cast<int>(N);
    a.eps = eps;
    a.one = static_cast<float>(offset);
    const bool wide = wide_rows(N, s, {{x, ldx}, {residual, ldres}, {gamma, 0}, {h, ldh}, {y, ldy}});
    a.same_phase = one_offset(s, {{h, ldh}, {y, ldy}});
    AddPlan p;
    p.dtype = dtype;
    p.drop = a.threshold != 0;
    p.mode = row_mode(wide, one_offset(s, {{x, ldx}, {residual, ldres}, {h, ldh}, {y, ldy}}));
    if (!fwd_shape(octets_of(N, dtype, wide), 8, p)) return RMSNORM_ERR_UNSUPPORTED;
    p.blocks = ceil_div(M, rows_per_block(p));
    return run(add_fwd_kernel(p), p, a, stream);
}

extern "C" size_t rmsnorm_add_bwd_workspace_size(int64_t M, int64_t N, rmsnorm_dtype dtype) {
    if (check_common(M, N, dtype, 0) != RMSNORM_OK || M == 0) return 0;
    int64_t units = 0;
    for (const RowMode mode : {kRowsAny, kRowsAligned, kRowsOnePhase})
        for (const bool drop : {false, true})
            for (const bool has_dh : {false, true}) {
                AddPlan p;
                if (add_bwd_plan(M, N, dtype, mode, drop, has_dh, p)) units = std::max(units, p.blocks);
            }
    (void)cudaGetLastError();
    return static_cast<size_t>(units) * static_cast<size_t>(workspace_pitch(N)) * sizeof(float);
}

extern "C" rmsnorm_status rmsnorm_add_bwd(const void* dy, int64_t lddy, const void* dh, int64_t lddh, const void* h,
                                          int64_t ldh, const void* gamma, const float* rstd, void* dx, int64_t lddx,
                                          void* dresidual, int64_t lddres, void* dgamma, int64_t M, int64_t N,
                                          rmsnorm_dtype dtype, int offset, float dropout_p, const uint64_t* rng,
                                          void* workspace, size_t workspace_bytes, rmsnorm_stream_t stream) {
    rmsnorm_status st = check_common(M, N, dtype, offset);
    if (st != RMSNORM_OK) return st;
    const size_t s = elem_bytes(dtype);
    if (!pitch_ok(lddy, N, M, s) || !pitch_ok(ldh, N, M, s) || (dh && !pitch_ok(lddh, N, M, s)) ||
        (dx && !pitch_ok(lddx, N, M, s)) || (dresidual && !pitch_ok(lddres, N, M, s)))
        return RMSNORM_ERR_SHAPE;
    AddArgs a = {};
    if (!check_dropout(dropout_p, rng, a, st)) return st;
    if (!dgamma) return RMSNORM_ERR_NULL;
    if (!aligned(dgamma, s)) return RMSNORM_ERR_ALIGN;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0)
        return launch_dgamma_reduce(dtype, nullptr, 0, static_cast<int>(N), workspace_pitch(N), dgamma, cs) == cudaSuccess
                   ? RMSNORM_OK
                   : RMSNORM_ERR_CUDA;
    if (!dy || !h || !gamma || !rstd || !workspace) return RMSNORM_ERR_NULL;
    if (!aligned(dy, s) || !aligned(dh, s) || !aligned(h, s) || !aligned(gamma, s) || !aligned(dx, s) ||
        !aligned(dresidual, s) || !aligned(rstd, 4) || !aligned(workspace, 16))
        return RMSNORM_ERR_ALIGN;
    if ((st = check_rng(a)) != RMSNORM_OK) return st;
    // without dropout dx and dresidual are equal, and may be one
    if (!distinct({dx, dgamma, workspace}) || !distinct({dresidual, dgamma, workspace}) ||
        (a.threshold && !distinct({dx, dresidual})) ||
        !same_rows(M, {dx, lddx}, {{dy, lddy}, {dh, lddh}, {h, ldh}, {gamma, 0}}) ||
        !same_rows(M, {dresidual, lddres}, {{dy, lddy}, {dh, lddh}, {h, ldh}, {gamma, 0}, {dx, lddx}}))
        return RMSNORM_ERR_ARG;
    AddPlan p;
    const bool wide = wide_rows(N, s, {{dy, lddy}, {dh, lddh}, {h, ldh}, {gamma, 0}, {dx, lddx}, {dresidual, lddres}});
    const RowMode mode =
        row_mode(wide, one_offset(s, {{dy, lddy}, {dh, lddh}, {h, ldh}, {dx, lddx}, {dresidual, lddres}}));
    if (!add_bwd_plan(M, N, dtype, mode, a.threshold != 0, dh != nullptr, p)) {
        (void)cudaGetLastError();
        return RMSNORM_ERR_CUDA;
    }
    a.ldws = workspace_pitch(N);
    if (workspace_bytes < static_cast<size_t>(p.blocks) * static_cast<size_t>(a.ldws) * sizeof(float))
        return RMSNORM_ERR_WORKSPACE;
    a.dy = dy;
    a.dh = dh;
    a.x = h;
    a.gamma = gamma;
    a.rstd = const_cast<float*>(rstd);
    a.dx = dx;
    a.dres = dresidual;
    a.ws = static_cast<float*>(workspace);
    a.lddy = lddy;
    a.lddh = lddh;
    a.ldx = ldh;
    a.lddx = lddx;
    a.lddres = lddres;
    a.M = M;
    a.N = static_cast<int>(N);
    a.one = static_cast<float>(offset);
    a.same_phase = one_offset(s, {{dx, lddx}, {dresidual, lddres}});
    if ((st = run(add_bwd_kernel(p), p, a, stream)) != RMSNORM_OK) return st;
    return launch_dgamma_reduce(dtype, a.ws, p.blocks, a.N, a.ldws, dgamma, cs) == cudaSuccess ? RMSNORM_OK
                                                                                              : RMSNORM_ERR_CUDA;
}

extern "C" rmsnorm_status rmsnorm_quant_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldres,
                                            const void* gamma, void* h, int64_t ldh, void* codes, int64_t ldcodes,
                                            float* scales, int64_t ldscales, int64_t M, int64_t N, float eps,
                                            rmsnorm_dtype dtype, int offset, int group, int pow2,
                                            rmsnorm_stream_t stream) {
    rmsnorm_status st = check_common(M, N, dtype, offset);
    if (st != RMSNORM_OK) return st;
    if (!std::isfinite(eps) || !(eps > 0.0f)) return RMSNORM_ERR_EPS;
    if ((group != 0 && group != 32 && group != 64 && group != 128) || (pow2 != 0 && pow2 != 1)) return RMSNORM_ERR_ARG;
    const size_t s = elem_bytes(dtype);
    if (!pitch_ok(ldx, N, M, s) || !pitch_ok(ldcodes, N, M, 1) || (residual && !pitch_ok(ldres, N, M, s)) ||
        (h && !pitch_ok(ldh, N, M, s)) || !pitch_ok(ldscales, group ? ceil_div(N, group) : 1, M, 4))
        return RMSNORM_ERR_SHAPE;
    if (M == 0) return RMSNORM_OK;
    if (!x || !gamma || !codes || !scales) return RMSNORM_ERR_NULL;
    // codes and scales are of other types than the inputs
    if (!distinct({h, codes, scales}) || !distinct({x, codes, scales}) || !distinct({residual, codes, scales}) ||
        !distinct({gamma, codes, scales}) || !same_rows(M, {h, ldh}, {{x, ldx}, {residual, ldres}, {gamma, 0}}))
        return RMSNORM_ERR_ARG;
    if (!aligned(x, s) || !aligned(residual, s) || !aligned(gamma, s) || !aligned(h, s) || !aligned(scales, 4))
        return RMSNORM_ERR_ALIGN;
    AddArgs a = {};
    a.x = x;
    a.res = residual;
    a.gamma = gamma;
    a.h = h;
    a.y = codes;
    a.scales = scales;
    a.ldx = ldx;
    a.ldres = ldres;
    a.ldh = ldh;
    a.ldy = ldcodes;
    a.ldscales = ldscales;
    a.M = M;
    a.N = static_cast<int>(N);
    a.inv_n = 1.0f / static_cast<float>(N);
    a.eps = eps;
    a.one = static_cast<float>(offset);
    a.group = group;
    a.group_shift = group == 128 ? 4 : group == 64 ? 3 : 2;
    a.pow2 = pow2;
    const bool wide = wide_rows(N, s, {{x, ldx}, {residual, ldres}, {gamma, 0}, {h, ldh}}) &&
                      wide_rows(N, 1, {{codes, ldcodes}});
    AddPlan p;
    p.dtype = dtype;
    // groups of columns want octets that start at column 0
    p.mode = row_mode(wide, group == 0 && one_offset(s, {{x, ldx}, {residual, ldres}, {h, ldh}}));
    const int64_t n = p.mode == kRowsOnePhase ? octets_of(N, dtype, false) : ceil_div(N, 8);
    if (!fwd_shape(n, 32, p)) return RMSNORM_ERR_UNSUPPORTED;
    p.blocks = ceil_div(M, rows_per_block(p));
    return run(quant_kernel(p), p, a, stream);
}

extern "C" rmsnorm_status rmsnorm_rope_fwd(const rmsnorm_rope_heads* sets, int nsets, const int64_t* positions,
                                           int64_t T, int64_t D, int64_t rotary_dim, const double* inv_freq,
                                           int interleaved, float mscale, float eps, rmsnorm_dtype dtype, int offset,
                                           rmsnorm_stream_t stream) {
    rmsnorm_status st = check_rope(nsets, T, D, rotary_dim, interleaved, mscale, eps, dtype, offset);
    if (st != RMSNORM_OK) return st;
    if (!sets) return RMSNORM_ERR_NULL;
    const size_t s = elem_bytes(dtype);
    RopeArgs a = {};
    bool wide = true;
    int64_t heads = 0;
    for (int i = 0; i < nsets; ++i) {
        const rmsnorm_rope_heads& q = sets[i];
        if (q.heads < 1 || q.heads > RMSNORM_ROPE_MAX_HEADS || !strides_ok(q.x_token, q.x_head, q.heads, T, D) ||
            !output_strides_ok(q.y_token, q.y_head, q.heads, T, D))
            return RMSNORM_ERR_SHAPE;
        heads += q.heads;
        if (T > 0 && (!q.x || !q.y)) return RMSNORM_ERR_NULL;
        if (!aligned(q.x, s) || !aligned(q.y, s) || !aligned(q.gamma, s)) return RMSNORM_ERR_ALIGN;
        RopeSet& t = a.set[i];
        t.x = q.x;
        t.gamma = q.gamma;
        t.y = q.y;
        t.x_token = q.x_token;
        t.x_head = q.x_head;
        t.y_token = q.y_token;
        t.y_head = q.y_head;
        t.heads = static_cast<int>(q.heads);
        wide = wide && rope_wide(t, s);
    }
    if (heads > RMSNORM_ROPE_MAX_HEADS) return RMSNORM_ERR_SHAPE;
    if (T == 0) return RMSNORM_OK;
    if (!outputs_ok(a, T, D, s, nsets)) return RMSNORM_ERR_ARG;
    if (!positions || !inv_freq) return RMSNORM_ERR_NULL;
    if (!aligned(positions, 8) || !aligned(inv_freq, 8)) return RMSNORM_ERR_ALIGN;
    a.nsets = nsets;
    a.heads = static_cast<int>(heads);
    a.pos = positions;
    a.inv_freq = inv_freq;
    a.T = T;
    a.D = static_cast<int>(D);
    a.R = static_cast<int>(rotary_dim);
    a.mscale = mscale;
    a.eps = eps;
    a.one = static_cast<float>(offset);
    RopePlan p;
    if ((st = rope_plan(a, dtype, interleaved, wide, false, p)) != RMSNORM_OK) return st;
    return rope_run(a, p, interleaved, false, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t rmsnorm_rope_bwd_workspace_size(int64_t T, int64_t heads, int64_t D, rmsnorm_dtype dtype) {
    if (check_common(T, D, dtype, 0) != RMSNORM_OK || D > RMSNORM_ROPE_MAX_D || T == 0 || heads < 1 ||
        heads > RMSNORM_ROPE_MAX_HEADS)
        return 0;
    int dev = 0;
    const int sms = current_sms(dev);
    // the backward's most blocks, a partial row each and set
    return static_cast<size_t>(RMSNORM_ROPE_MAX_SETS) * static_cast<size_t>(std::min<int64_t>(T * heads, int64_t(sms) * 8)) *
           static_cast<size_t>(workspace_pitch(D)) * sizeof(float);
}

extern "C" rmsnorm_status rmsnorm_rope_bwd(const rmsnorm_rope_heads_bwd* sets, int nsets, const int64_t* positions,
                                           int64_t T, int64_t D, int64_t rotary_dim, const double* inv_freq,
                                           int interleaved, float mscale, float eps, rmsnorm_dtype dtype, int offset,
                                           void* workspace, size_t workspace_bytes, rmsnorm_stream_t stream) {
    rmsnorm_status st = check_rope(nsets, T, D, rotary_dim, interleaved, mscale, eps, dtype, offset);
    if (st != RMSNORM_OK) return st;
    if (!sets) return RMSNORM_ERR_NULL;
    const size_t s = elem_bytes(dtype);
    RopeArgs a = {};
    bool wide = true;
    int64_t heads = 0;
    bool weights = false;
    for (int i = 0; i < nsets; ++i) {
        const rmsnorm_rope_heads_bwd& q = sets[i];
        if (q.heads < 1 || q.heads > RMSNORM_ROPE_MAX_HEADS || !strides_ok(q.dy_token, q.dy_head, q.heads, T, D) ||
            (q.gamma && !strides_ok(q.x_token, q.x_head, q.heads, T, D)) ||
            !output_strides_ok(q.dx_token, q.dx_head, q.heads, T, D))
            return RMSNORM_ERR_SHAPE;
        heads += q.heads;
        weights = weights || q.gamma;
        if ((T > 0 && (!q.dy || !q.dx || (q.gamma && !q.x))) || (q.gamma && !q.dgamma)) return RMSNORM_ERR_NULL;
        if (!aligned(q.dy, s) || !aligned(q.dx, s) || !aligned(q.gamma, s) || (q.gamma && (!aligned(q.x, s) || !aligned(q.dgamma, s))))
            return RMSNORM_ERR_ALIGN;
        RopeSet& t = a.set[i];
        t.dy = q.dy;
        t.gamma = q.gamma;
        t.y = q.dx;
        t.dy_token = q.dy_token;
        t.dy_head = q.dy_head;
        if (q.gamma) {
            t.x = q.x;
            t.x_token = q.x_token;
            t.x_head = q.x_head;
        }
        t.y_token = q.dx_token;
        t.y_head = q.dx_head;
        t.heads = static_cast<int>(q.heads);
        wide = wide && rope_wide(t, s);
    }
    if (heads > RMSNORM_ROPE_MAX_HEADS) return RMSNORM_ERR_SHAPE;
    if (nsets == 2 && sets[0].gamma && sets[1].gamma && sets[0].dgamma == sets[1].dgamma) return RMSNORM_ERR_ARG;
    if (T > 0 && !outputs_ok(a, T, D, s, nsets)) return RMSNORM_ERR_ARG;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    a.nsets = nsets;
    a.heads = static_cast<int>(heads);
    a.pos = positions;
    a.inv_freq = inv_freq;
    a.T = T;
    a.D = static_cast<int>(D);
    a.R = static_cast<int>(rotary_dim);
    a.mscale = mscale;
    a.eps = eps;
    a.one = static_cast<float>(offset);
    if (T > 0) {
        if (!positions || !inv_freq || (weights && !workspace)) return RMSNORM_ERR_NULL;
        if (!aligned(positions, 8) || !aligned(inv_freq, 8) || !aligned(workspace, 16)) return RMSNORM_ERR_ALIGN;
        RopePlan p;
        if ((st = rope_plan(a, dtype, interleaved, wide, true, p)) != RMSNORM_OK) return st;
        const size_t need = static_cast<size_t>(nsets) * static_cast<size_t>(a.units) * static_cast<size_t>(a.ldws) * sizeof(float);
        if (weights && workspace_bytes < need) return RMSNORM_ERR_WORKSPACE;
        a.ws = static_cast<float*>(workspace);
        if ((st = rope_run(a, p, interleaved, true, cs)) != RMSNORM_OK) return st;
    }
    // a set's partials are a plane of `units` rows; two sets take one launch
    const int64_t plane = a.units * a.ldws;
    if (nsets == 2 && sets[0].gamma && sets[1].gamma)
        return launch_dgamma_reduce(dtype, a.ws, a.units, a.D, workspace_pitch(D), sets[0].dgamma, cs, sets[1].dgamma) ==
                       cudaSuccess
                   ? RMSNORM_OK
                   : RMSNORM_ERR_CUDA;
    for (int i = 0; i < nsets; ++i)
        if (sets[i].gamma && launch_dgamma_reduce(dtype, a.ws ? a.ws + i * plane : nullptr, a.units, a.D, workspace_pitch(D),
                                                  sets[i].dgamma, cs) != cudaSuccess)
            return RMSNORM_ERR_CUDA;
    return RMSNORM_OK;
}
