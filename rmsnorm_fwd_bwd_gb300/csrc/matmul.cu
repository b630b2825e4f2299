// matmul.cu -- products of e4m3 codes with scales: y = (a sa) (b sb)^T + bias.
//
// a is [M, K] with a scale per row and 128 columns (or per row), b [N, K] with one per
// block of 128 x 128. Over one block of 128 columns both scales of an element of y are
// constants, so
//     y[m, n] = sum over blocks j of sa[m, j] * sb[n / 128, j] * (a_j b_j^T)[m, n].
// The inner products of a block, 128 products of codes, are summed by the tensor cores in
// fp32; the sum over blocks is taken in fp32 registers, by one multiply-add per element and
// block (two of them in one packed instruction).
//
// Three kernels. matmul_pair: pairs of blocks on tiles of 256 x 256, a thread to a row of the
// accumulator. matmul_wide: single blocks on tiles of 128 x 128. matmul_thin, for few rows
// of a: the operands change places, a tile is 128 rows of b and 16 to 128 of a, and the blocks of a
// cluster share K. In all of them one thread keeps a ring of tiles full by TMA, one issues
// the matrix instructions into one of several accumulators in tensor memory, and warps of four
// add finished ones up meanwhile. Rows off 16 bytes, which TMA does not take, are loaded
// by three warps in words that are shifted together.
#include "octet.cuh"
#include "serving.h"
#include "tcgen05.cuh"

namespace rmsnorm {
namespace {

constexpr int kMostSplit = kMatmulMostSplit;
constexpr int kTileBytes = 128 * kTileK;  // 128 rows

constexpr int kWideStages = 6, kPairStages = 6;
// Two blocks to an SM, but for 128 rows of a, which leave room for one.
constexpr int thin_blocks(int n) { return n < 128 ? 2 : 1; }
constexpr int thin_stages(int n) { return n < 32 ? 5 : n < 128 ? 4 : 6; }
// Accumulators in tensor memory that are under way.
constexpr int kWideBuffers = 4, kPairBuffers = 2;
constexpr int kThinBuffers = 4;
constexpr int thin_columns(int n) { return kThinBuffers * n; }

// 16 codes of a row from column k on, any alignment; those from `left` on are zero. Only
// 16-byte words that hold a code of the row are read.
__device__ __forceinline__ uint4 codes16(const uint8_t* p, int64_t left) {
    uint32_t s[9];
    const uint32_t sh = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15);
    const uint4* q = reinterpret_cast<const uint4*>(p - sh);
    uint4 v = make_uint4(0u, 0u, 0u, 0u), u = v;
    if (left > 0) v = q[0];
    if (static_cast<int64_t>(sh) + (left < 16 ? left : 16) > 16) u = q[1];
    s[0] = v.x; s[1] = v.y; s[2] = v.z; s[3] = v.w;
    s[4] = u.x; s[5] = u.y; s[6] = u.z; s[7] = u.w;
    s[8] = 0u;
    if (sh & 8u) {
#pragma unroll
        for (int i = 0; i < 6; ++i) s[i] = s[i + 2];
    }
    if (sh & 4u) {
#pragma unroll
        for (int i = 0; i < 6; ++i) s[i] = s[i + 1];
    }
    const uint32_t bits = 8u * (sh & 3u);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = __funnelshift_r(s[i], s[i + 1], bits);
        const int64_t n = left - 4 * i;  // codes of this word
        if (n < 4) w[i] = n <= 0 ? 0u : w[i] & ((1u << (8 * static_cast<int>(n))) - 1u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The threads that load tiles of rows off 16 bytes: with those that add up and the one that
// issues they are eight warps, which leaves each all the registers that a thread can have.
constexpr int kLoaders = 96;

// ROWS rows of a tile from row r0 and column k0 on, into swizzled shared memory, by kLoaders
// threads: rows and columns outside of the matrix are zero.
template <int ROWS>
__device__ __forceinline__ void load_tile(uint32_t dst, const uint8_t* base, int64_t ld, int64_t r0, int64_t rows, int k0,
                                          int K, int thread) {
    constexpr int BATCH = 4;
#pragma unroll 1
    for (int first = thread; first < ROWS * 8; first += kLoaders * BATCH) {
        uint4 v[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int at = first + kLoaders * i, row = at >> 3, k = k0 + (at & 7) * 16;
            const bool in = at < ROWS * 8 && r0 + row < rows;
            v[i] = codes16(base + (in ? (r0 + row) * ld : 0) + (in ? k : 0), in ? static_cast<int64_t>(K) - k : 0);
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int at = first + kLoaders * i, row = at >> 3, c = at & 7;
            if (at < ROWS * 8)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + row * kTileK + ((c ^ (row & 7)) << 4)),
                             "r"(v[i].x), "r"(v[i].y), "r"(v[i].z), "r"(v[i].w)
                             : "memory");
        }
    }
}

// Position in a ring of N places: index and phase.
template <int N> struct Ring {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) {
            at = 0;
            phase ^= 1u;
        }
    }
};

// The barriers of a block: ring places filled and emptied, accumulators filled and emptied,
// and one for the instructions under way when a wait has given up.
template <int STAGES, int BUFFERS> struct Bars {
    uint64_t full[STAGES], empty[STAGES], done[BUFFERS], taken[BUFFERS], drain;
    uint32_t tmem;
    __device__ __forceinline__ void init(int producers, int takers) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(smem_u32(&full[i]), producers);
            mbar_init(smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < BUFFERS; ++i) {
            mbar_init(smem_u32(&done[i]), 1);
            mbar_init(smem_u32(&taken[i]), takers);
        }
        mbar_init(smem_u32(&drain), 1);
        fence_mbar_init();
    }
};

// The warp that issues matrix instructions: `blocks` blocks of K through the ring (X rows by Y
// rows, X's tile first in a stage of BYTES) into the accumulators in turn. PAIR: for both blocks
// of a cluster, X of 256 rows. The loop is the whole warp's, see elect_lane (16384 x 8192 x 8192
// 1110 us with a loop of one thread).
template <int STAGES, int BUFFERS, int Y, bool PAIR>
__device__ __forceinline__ void issue(Bars<STAGES, BUFFERS>& bars, uint32_t tiles, uint32_t tmem, int64_t blocks, uint32_t* err) {
    constexpr uint32_t kStage = PAIR ? 2 * kTileBytes : kTileBytes + Y * kTileK;
    constexpr uint32_t idesc = e4m3_idesc(PAIR ? 256 : 128, Y);
    const uint64_t x0 = tile_desc(tiles), y0 = tile_desc(tiles + kTileBytes);
    const uint32_t full = smem_u32(bars.full), empty = smem_u32(bars.empty), done = smem_u32(bars.done),
                   taken = smem_u32(bars.taken);
    Ring<STAGES> s;
    Ring<BUFFERS> b;
    for (int64_t i = 0; i < blocks; ++i) {
        const bool ok = mbar_wait_bounded(taken + 8 * b.at, b.phase ^ 1u, err) && mbar_wait_bounded(full + 8 * s.at, s.phase, err);
        if (!__all_sync(0xffffffffu, ok)) {
            if (elect_lane()) {
                const uint32_t drain = smem_u32(&bars.drain);
                if (PAIR) mma_commit_pair(drain);
                else mma_commit(drain);
            }
            mbar_wait_bounded(smem_u32(&bars.drain), 0, err);
            return;
        }
        tmem_fence_after();
        if (elect_lane()) {
            const uint64_t x = x0 + s.at * (kStage >> 4), y = y0 + s.at * (kStage >> 4);
            const uint32_t d = tmem + b.at * Y;
#pragma unroll
            for (int k = 0; k < kTileK / 32; ++k) {
                if (PAIR) mma_e4m3_pair(d, x + 2 * k, y + 2 * k, idesc, k > 0);
                else mma_e4m3(d, x + 2 * k, y + 2 * k, idesc, k > 0);
            }
            if (PAIR) {
                mma_commit_pair(empty + 8 * s.at);
                mma_commit_pair(done + 8 * b.at);
            } else {
                mma_commit(empty + 8 * s.at);
                mma_commit(done + 8 * b.at);
            }
        }
        __syncwarp();
        s.next();
        b.next();
    }
}

// After a wait that gave up: the tiles that are still on their way, `issued` in all.
template <int STAGES, int BUFFERS>
__device__ __forceinline__ void drain_tiles(Bars<STAGES, BUFFERS>& bars, int64_t issued, uint32_t* err) {
    for (int64_t i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
        mbar_wait_bounded(smem_u32(&bars.full[i % STAGES]), static_cast<uint32_t>(i / STAGES & 1), err);
}

// A finished accumulator's columns [0, C) of this thread's row, each times its factor (given for
// four columns), added to
// acc; `arrive` gives it back as soon as it is in registers. Single multiply-adds: packed pairs
// want their operands in pairs of registers, where the loads do not put them, and cost as many
// moves (16384 x 8192 x 8192 1375 us with them, 1100 without).
template <int C, class Arrive, class Factor>
__device__ __forceinline__ void add_up(uint32_t tmem, float (&acc)[C], Arrive&& arrive, Factor&& factor) {
    constexpr int W = C < 32 ? 16 : 32;
    uint32_t t[2][W];
    tmem_load(tmem, t[0]);
#pragma unroll
    for (int c = 0; c < C; c += W) {
        uint32_t(&now)[W] = t[(c / W) & 1];
        tmem_wait_loads(now);
        if (c + W < C) {
            tmem_load(tmem + c + W, t[(c / W + 1) & 1]);
        } else {
            tmem_fence_before();
            __syncwarp();
            if ((threadIdx.x & 31) == 0) arrive();
        }
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const float4 f = factor(c + i);
            acc[c + i] = fmaf(__uint_as_float(now[i]), f.x, acc[c + i]);
            acc[c + i + 1] = fmaf(__uint_as_float(now[i + 1]), f.y, acc[c + i + 1]);
            acc[c + i + 2] = fmaf(__uint_as_float(now[i + 2]), f.z, acc[c + i + 2]);
            acc[c + i + 3] = fmaf(__uint_as_float(now[i + 3]), f.w, acc[c + i + 3]);
        }
    }
}

// The tile of turn `t`: bands of up to 16 tiles of a, and within a band b's tiles one after the
// other, so that the blocks that run at a time share both in the L2.
__device__ __forceinline__ void tile_at(const MatmulArgs& a, int64_t t, int& m, int& n) {
    constexpr int kBand = 16;
    const int64_t per_band = static_cast<int64_t>(kBand) * a.n_tiles;
    const int band = static_cast<int>(t / per_band);
    const int rows = min(kBand, a.m_tiles - band * kBand);
    const int rest = static_cast<int>(t - band * per_band);
    n = rest / rows;
    m = band * kBand + rest - n * rows;
}

// A warp that adds up 128 columns of an accumulator (from its column `shift` on) for the tiles
// from `first` on, every `step`th, and stores them. A tile has `rows` rows, of which this
// block has those from `row_shift` on.
template <int DT, int BN, int BUFFERS, class Done, class Taken>
__device__ __forceinline__ void add_tiles(const MatmulArgs& a, uint32_t tmem, int shift, int64_t first, int64_t step, int rows,
                                          int row_shift, Done&& done, Taken&& taken) {
    constexpr int EB = Elem<DT>::kBytes, V = Elem<DT>::kVec;
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const uint32_t mine = tmem + (static_cast<uint32_t>(quarter) << 21) + shift;
    const int64_t all = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    Ring<BUFFERS> b;
    bool ok = true;
    for (int64_t t = first; t < all; t += step) {
        __syncwarp();
        if (!ok) break;  // in all lanes
        int m, n;
        tile_at(a, t, m, n);
        const int64_t row = static_cast<int64_t>(m) * rows + row_shift + quarter * 32 + lane;
        const int col = n * BN + shift;
        const bool live = row < a.M && col < a.N;
        const float* sa = a.sa + (live ? row * a.ldsa : 0);
        const float* sb = a.sb + (live ? (col >> 7) * a.ldsb : 0);
        float acc[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) acc[i] = 0.f;
        float fa = live ? sa[0] : 0.f, fb = live ? sb[0] : 0.f;
        for (int kb = 0; kb < a.kblocks; ++kb) {
            const float f = fa * fb;
            if (live && kb + 1 < a.kblocks) {
                if (!a.per_row) fa = sa[kb + 1];
                fb = sb[kb + 1];
            }
            ok = mbar_wait_bounded(done(b.at), b.phase, a.err);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tmem_fence_after();
            add_up<128>(mine + b.at * BN, acc, [&] { taken(b.at); }, [&](int) { return make_float4(f, f, f, f); });
            b.next();
        }
        __syncwarp();
        if (!ok || !live) continue;
        char* out = static_cast<char*>(a.y) + (row * a.ldy + col) * EB;
#pragma unroll
        for (int c = 0; c < 128; c += V) {
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = acc[c + i];
            if (a.bias) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (col + c + i < a.N) v[i] += Elem<DT>::ld(a.bias, col + c + i);
            }
            if (a.wide_y && col + c + V <= a.N) {
                *reinterpret_cast<uint4*>(out + c * EB) = Elem<DT>::pack(v);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (col + c + i < a.N) Elem<DT>::st(out, c + i, v[i]);
            }
        }
    }
}

constexpr int wide_threads(bool tma) { return 160 + (tma ? 32 : kLoaders); }
constexpr int thin_threads(bool tma) { return 160 + (tma ? 32 : kLoaders); }
constexpr int kPairThreads = 384;

template <int DT, bool TMA>
__global__ void __launch_bounds__(wide_threads(TMA), 1)
    matmul_wide(const MatmulArgs a, const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap) {
    constexpr int STAGES = kWideStages, BUFFERS = kWideBuffers;
    constexpr uint32_t kStage = 2 * kTileBytes;
    extern __shared__ char dynamic[];
    __shared__ Bars<STAGES, BUFFERS> bars;
    const uint32_t tiles = (smem_u32(dynamic) + 1023u) & ~1023u;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform to the compiler
    constexpr int kIssuer = 4, kProducer = 5;
    if (warp == kIssuer) tmem_alloc(smem_u32(&bars.tmem), 512);
    if (threadIdx.x == 0) bars.init(TMA ? 1 : kLoaders, 4);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = bars.tmem;
    griddep_wait();
    const int64_t all = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    if (warp >= kProducer) {
        Ring<STAGES> s;
        int64_t issued = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; ok && t < all; t += gridDim.x) {
            int m, n;
            tile_at(a, t, m, n);
            for (int kb = 0; kb < a.kblocks; ++kb) {
                ok = mbar_wait_bounded(smem_u32(bars.empty) + 8 * s.at, s.phase ^ 1u, a.err);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const uint32_t dst = tiles + s.at * kStage, full = smem_u32(bars.full) + 8 * s.at;
                if constexpr (TMA) {
                    if (elect_lane()) {
                        mbar_arrive_expect_tx(full, kStage);
                        tile_g2s(dst, &amap, kb * kTileK, m * 128, full);
                        tile_g2s(dst + kTileBytes, &bmap, kb * kTileK, n * 128, full);
                    }
                    __syncwarp();
                } else {
                    const int thread = threadIdx.x - kProducer * 32;
                    load_tile<128>(dst, a.a, a.lda, static_cast<int64_t>(m) * 128, a.M, kb * kTileK, a.K, thread);
                    load_tile<128>(dst + kTileBytes, a.b, a.ldb, static_cast<int64_t>(n) * 128, a.N, kb * kTileK, a.K, thread);
                    fence_proxy_async_smem();
                    mbar_arrive(full);
                }
                ++issued;
                s.next();
            }
        }
        if (TMA && !ok) drain_tiles(bars, issued, a.err);
    } else if (warp == kIssuer) {
        const int64_t mine = all > blockIdx.x ? (all - blockIdx.x - 1) / gridDim.x + 1 : 0;
        issue<STAGES, BUFFERS, 128, false>(bars, tiles, tmem, mine * a.kblocks, a.err);
    } else {
        add_tiles<DT, 128, BUFFERS>(a, tmem, 0, blockIdx.x, gridDim.x, 128, 0, [&](int i) { return smem_u32(&bars.done[i]); },
                                    [&](int i) { mbar_arrive(smem_u32(&bars.taken[i])); });
    }
    griddep_launch_dependents();
    tmem_fence_before();
    __syncthreads();
    if (warp == kIssuer) tmem_free(tmem, 512);
}

// Pairs of blocks (clusters of two): a tile of 256 rows of a by 256 of b, for which each block
// loads 128 rows of both; the tensor cores of both work on one instruction, from one thread
// of the first block, and read the other block's half of b from its shared memory. Two
// thirds of the L2's traffic of blocks on their own.
template <int DT>
__global__ void __launch_bounds__(kPairThreads, 1)
    matmul_pair(const MatmulArgs a, const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap) {
    constexpr int STAGES = kPairStages, BUFFERS = kPairBuffers;
    constexpr uint32_t kStage = 2 * kTileBytes;
    extern __shared__ char dynamic[];
    __shared__ Bars<STAGES, BUFFERS> bars;
    const uint32_t tiles = (smem_u32(dynamic) + 1023u) & ~1023u;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform to the compiler
    const int rank = static_cast<int>(cluster_rank());
    constexpr int kIssuer = 8, kProducer = 9;
    if (warp == kIssuer) tmem_alloc_pair(smem_u32(&bars.tmem), 512);
    // an accumulator is taken when the 8 warps of both blocks have it
    if (threadIdx.x == 0) bars.init(1, 16);
    __syncwarp();
    tmem_fence_before();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = bars.tmem;
    griddep_wait();
    const int64_t all = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
    // the 384 threads have 168 registers at first: the 8 warps that add up take 232, the others
    // keep 40
    if (warp >= kIssuer) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == kProducer) {
            Ring<STAGES> s;
            int64_t issued = 0;
            bool ok = true;
            // the first block's barriers count both blocks' tiles
            const uint32_t both = dsmem_map(smem_u32(bars.full), 0);
            for (int64_t t = first; ok && t < all; t += step) {
                int m, n;
                tile_at(a, t, m, n);
                for (int kb = 0; kb < a.kblocks; ++kb) {
                    ok = mbar_wait_bounded(smem_u32(bars.empty) + 8 * s.at, s.phase ^ 1u, a.err);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    if (elect_lane()) {
                        const uint32_t dst = tiles + s.at * kStage;
                        if (rank == 0) mbar_arrive_expect_tx(smem_u32(bars.full) + 8 * s.at, 2 * kStage);
                        tile_g2s_pair(dst, &amap, kb * kTileK, m * 256 + rank * 128, both + 8 * s.at);
                        tile_g2s_pair(dst + kTileBytes, &bmap, kb * kTileK, n * 256 + rank * 128, both + 8 * s.at);
                    }
                    __syncwarp();
                    ++issued;
                    s.next();
                }
            }
            if (!ok && rank == 0) drain_tiles(bars, issued, a.err);
        } else if (warp == kIssuer && rank == 0) {
            const int64_t mine = all > first ? (all - first - 1) / step + 1 : 0;
            issue<STAGES, BUFFERS, 256, true>(bars, tiles, tmem, mine * a.kblocks, a.err);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        add_tiles<DT, 256, BUFFERS>(a, tmem, (warp >> 2) * 128, first, step, 256, rank * 128,
                                    [&](int i) { return smem_u32(&bars.done[i]); },
                                    [&](int i) { mbar_arrive_cluster(dsmem_map(smem_u32(&bars.taken[i]), 0)); });
    }
    griddep_launch_dependents();
    tmem_fence_before();
    __syncwarp();
    cluster_sync();  // no block leaves before the other's instructions and arrivals
    if (warp == kIssuer) tmem_free_pair(tmem, 512);
}

// Few rows of a: 128 rows of b are the accumulator's lanes, NT rows of a its columns. The
// blocks of a cluster take a part of K each; their sums meet in shared memory and are
// added in the blocks' order, so that the result does not depend on who was first.
// Blocks of K whose factors lie in shared memory at a time.
constexpr int kFactorBlocks = 16;

template <int DT, int NT, bool TMA>
__global__ void __launch_bounds__(thin_threads(TMA), thin_blocks(NT))
    matmul_thin(const MatmulArgs a, const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap) {
    constexpr int STAGES = thin_stages(NT), BUFFERS = kThinBuffers;
    constexpr uint32_t kStage = kTileBytes + NT * kTileK;
    extern __shared__ char dynamic[];
    __shared__ Bars<STAGES, BUFFERS> bars;
    __shared__ alignas(16) float factors[2][kFactorBlocks][NT + 4];
    const uint32_t base = smem_u32(dynamic), tiles = (base + 1023u) & ~1023u;
    float* sums = reinterpret_cast<float*>(dynamic + (tiles - base));  // [NT][128], where the tiles were
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform to the compiler
    constexpr int kIssuer = 4, kProducer = 5;
    if (warp == kIssuer) tmem_alloc(smem_u32(&bars.tmem), thin_columns(NT));
    if (threadIdx.x == 0) bars.init(TMA ? 1 : kLoaders, 4);
    if (TMA && threadIdx.x == kProducer * 32) {
        prefetch_map(&amap);
        prefetch_map(&bmap);
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = bars.tmem;
    griddep_wait();
    griddep_launch_dependents();
    const int split = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    const int tile = static_cast<int>(blockIdx.x) / split;
    const int m = tile / a.n_tiles, n = tile - m * a.n_tiles;
    const int64_t t0 = static_cast<int64_t>(m) * NT;
    const int from = static_cast<int>(static_cast<int64_t>(a.kblocks) * rank / split);
    const int to = static_cast<int>(static_cast<int64_t>(a.kblocks) * (rank + 1) / split);
    constexpr int EB = Elem<DT>::kBytes;
    const int col = n * 128 + threadIdx.x;  // of y, for the threads that add up
    const int rows = static_cast<int>(min(static_cast<int64_t>(NT), a.M - t0));
    bool ok = true;
    if (warp >= kProducer) {
        Ring<STAGES> s;
        int64_t issued = 0;
        for (int kb = from; kb < to; ++kb) {
            ok = mbar_wait_bounded(smem_u32(bars.empty) + 8 * s.at, s.phase ^ 1u, a.err);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            const uint32_t dst = tiles + s.at * kStage, full = smem_u32(bars.full) + 8 * s.at;
            if constexpr (TMA) {
                if (elect_lane()) {
                    mbar_arrive_expect_tx(full, kStage);
                    tile_g2s(dst, &bmap, kb * kTileK, n * 128, full);
                    tile_g2s(dst + kTileBytes, &amap, kb * kTileK, m * NT, full);
                }
                __syncwarp();
            } else {
                const int thread = threadIdx.x - kProducer * 32;
                load_tile<128>(dst, a.b, a.ldb, static_cast<int64_t>(n) * 128, a.N, kb * kTileK, a.K, thread);
                load_tile<NT>(dst + kTileBytes, a.a, a.lda, t0, a.M, kb * kTileK, a.K, thread);
                fence_proxy_async_smem();
                mbar_arrive(full);
            }
            ++issued;
            s.next();
        }
        if (TMA && !ok) drain_tiles(bars, issued, a.err);
        __syncwarp();
    } else if (warp == kIssuer) {
        issue<STAGES, BUFFERS, NT, false>(bars, tiles, tmem, to - from, a.err);
        __syncwarp();
    } else {
        const uint32_t mine = tmem + (static_cast<uint32_t>(warp) << 21);
        // factors of kFactorBlocks blocks at a time: a thread loads those of block `fb` of a chunk for
        // the rows fr, fr + 8, ..., a chunk ahead
        constexpr int E = kFactorBlocks * NT / 128;
        const int fb = threadIdx.x % kFactorBlocks, fr = threadIdx.x / kFactorBlocks;
        const float* sa = a.sa + (a.per_row ? 0 : fb);
        const float* sb = a.sb + n * a.ldsb + fb;
        float fv[E], fs;
        const auto fetch = [&](int kb) {
            const bool in = kb + fb < to;
            fs = in ? sb[kb] : 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int row = fr + 8 * i;
                fv[i] = in && row < rows ? sa[(t0 + row) * a.ldsa + (a.per_row ? 0 : kb)] : 0.f;
            }
        };
        const auto keep = [&](int which) {
#pragma unroll
            for (int i = 0; i < E; ++i) factors[which][fb][fr + 8 * i] = fv[i] * fs;
            named_barrier_sync(1, 128);
        };
        float acc[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i] = 0.f;
        Ring<BUFFERS> b;
        fetch(from);
        keep(0);
        int which = 0;
        for (int k0 = from; k0 < to; k0 += kFactorBlocks, which ^= 1) {
            const bool more = k0 + kFactorBlocks < to;
            if (more) fetch(k0 + kFactorBlocks);
            const int n_blocks = min(kFactorBlocks, to - k0);
            for (int i = 0; i < n_blocks; ++i) {
                ok = mbar_wait_bounded(smem_u32(bars.done) + 8 * b.at, b.phase, a.err) && ok;
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tmem_fence_after();
                const float* f = factors[which][i];
                add_up<NT>(mine + b.at * NT, acc, [&] { mbar_arrive(smem_u32(bars.taken) + 8 * b.at); },
                           [&](int c) { return *reinterpret_cast<const float4*>(f + c); });
                b.next();
            }
            // (where a wait gave up the others go on meeting at the barrier)
            if (more) keep(which ^ 1);
        }
        const float bias = a.bias && col < a.N ? Elem<DT>::ld(a.bias, col) : 0.f;
        if (split == 1) {
            if (ok && col < a.N) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (j < rows) Elem<DT>::st(static_cast<char*>(a.y) + ((t0 + j) * a.ldy + col) * EB, 0, acc[j] + bias);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NT; ++j) sums[j * 128 + threadIdx.x] = acc[j];
        }
    }
    __syncwarp();
    if (split > 1) {
        cluster_sync();
        if (warp < 4 && ok && col < a.N) {
            const float bias = a.bias ? Elem<DT>::ld(a.bias, col) : 0.f;
            const uint32_t at = smem_u32(sums) + threadIdx.x * 4;
            for (int j = rank; j < rows; j += split) {
                float part[kMostSplit], v = 0.f;
#pragma unroll
                for (int r = 0; r < kMostSplit; ++r) part[r] = r < split ? dsmem_ld_f32(dsmem_map(at + j * 512, r)) : 0.f;
#pragma unroll
                for (int r = 0; r < kMostSplit; ++r) v += part[r];
                Elem<DT>::st(static_cast<char*>(a.y) + ((t0 + j) * a.ldy + col) * EB, 0, v + bias);
            }
        }
        __syncwarp();
        cluster_sync();
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kIssuer) tmem_free(tmem, thin_columns(NT));
}

template <int DT, bool TMA> const void* kernel_for(const MatmulPlan& p) {
    if (p.how == kMatmulPair) return TMA ? reinterpret_cast<const void*>(&matmul_pair<DT>) : nullptr;
    if (p.how == kMatmulWide) return reinterpret_cast<const void*>(&matmul_wide<DT, TMA>);
    switch (p.n) {
    case 16: return reinterpret_cast<const void*>(&matmul_thin<DT, 16, TMA>);
    case 32: return reinterpret_cast<const void*>(&matmul_thin<DT, 32, TMA>);
    case 64: return reinterpret_cast<const void*>(&matmul_thin<DT, 64, TMA>);
    case 128: return reinterpret_cast<const void*>(&matmul_thin<DT, 128, TMA>);
    default: return nullptr;
    }
}

}  // namespace

const void* matmul_kernel(const MatmulPlan& p) {
    switch (p.dtype) {
    case kF32: return p.tma ? kernel_for<kF32, true>(p) : kernel_for<kF32, false>(p);
    case kF16: return p.tma ? kernel_for<kF16, true>(p) : kernel_for<kF16, false>(p);
    case kBF16: return p.tma ? kernel_for<kBF16, true>(p) : kernel_for<kBF16, false>(p);
    default: return nullptr;
    }
}

void matmul_shape(MatmulPlan& p) {
    const bool thin = p.how == kMatmulThin;
    const int stages = thin ? thin_stages(p.n) : p.how == kMatmulWide ? kWideStages : kPairStages;
    p.threads = thin ? thin_threads(p.tma) : p.how == kMatmulWide ? wide_threads(p.tma) : kPairThreads;
    p.smem = 1024 + static_cast<size_t>(stages) * (kTileBytes + (thin ? p.n * kTileK : kTileBytes));
}

}  // namespace rmsnorm
