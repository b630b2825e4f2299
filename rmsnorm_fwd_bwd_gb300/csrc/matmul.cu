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
// Two kernels. matmul_wide: a tile of 128 rows of a (a thread's row of the accumulator) and
// 128 or 256 of b, persistent blocks. matmul_thin, for few rows of a: the operands change places, a
// tile is 128 rows of b and 16 to 128 of a, and the blocks of a cluster share K. In both one
// thread keeps a ring of tiles full by TMA, one issues the matrix instructions into one of
// several accumulators in tensor memory, and warps of four add finished ones up meanwhile.
// Rows off 16 bytes, which TMA does not take, are loaded by four warps in words
// that are shifted together.
#include "octet.cuh"
#include "serving.h"
#include "tcgen05.cuh"

namespace rmsnorm {
namespace {

constexpr int kTileBytes = 128 * kTileK;  // 128 rows

constexpr int wide_stages(int n) { return n == 256 ? 4 : 6; }
constexpr int thin_stages(int n) { return n <= 32 ? 9 : n == 64 ? 8 : 6; }
// Accumulators in tensor memory that are under way.
constexpr int wide_buffers(int n) { return 512 / n; }
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

// The thread that issues matrix instructions: `blocks` blocks of K through the ring (X rows
// by Y rows, X's tile first in a stage) into the accumulators in turn.
template <int STAGES, int BUFFERS, int Y>
__device__ __forceinline__ void issue(Bars<STAGES, BUFFERS>& bars, uint32_t tiles, uint32_t tmem, int64_t blocks, uint32_t* err) {
    constexpr uint32_t kStage = kTileBytes + Y * kTileK;
    constexpr uint32_t idesc = e4m3_idesc(128, Y);
    Ring<STAGES> s;
    Ring<BUFFERS> b;
    for (int64_t i = 0; i < blocks; ++i) {
        if (!mbar_wait_bounded(smem_u32(&bars.taken[b.at]), b.phase ^ 1u, err) ||
            !mbar_wait_bounded(smem_u32(&bars.full[s.at]), s.phase, err)) {
            mma_commit(smem_u32(&bars.drain));
            mbar_wait_bounded(smem_u32(&bars.drain), 0, err);
            return;
        }
        tmem_fence_after();
        const uint64_t x = tile_desc(tiles + s.at * kStage), y = tile_desc(tiles + s.at * kStage + kTileBytes);
#pragma unroll
        for (int k = 0; k < kTileK / 32; ++k) mma_e4m3(tmem + b.at * Y, x + 2 * k, y + 2 * k, idesc, k > 0);
        mma_commit(smem_u32(&bars.empty[s.at]));
        mma_commit(smem_u32(&bars.done[b.at]));
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

// A finished accumulator's columns [0, C) of this thread's row, times f (two columns' factors
// to a word, or one factor for all), added to acc.
template <int C, class Factor>
__device__ __forceinline__ void add_up(uint32_t tmem, uint64_t (&acc)[C / 2], uint32_t taken, Factor&& factor) {
    constexpr int W = C < 32 ? 16 : 32;
#pragma unroll
    for (int c = 0; c < C; c += W) {
        uint32_t t[W];
        tmem_load(tmem + c, t);
        tmem_wait_loads();
        if (c + W == C) {
            tmem_fence_before();
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(taken);
        }
#pragma unroll
        for (int i = 0; i < W; i += 2)
            acc[(c + i) / 2] = f2_fma(f2_pack(__uint_as_float(t[i]), __uint_as_float(t[i + 1])), factor(c + i), acc[(c + i) / 2]);
    }
}

// The tile of a persistent block's turn `t`: bands of up to 16 tiles of a, and within a band
// b's tiles one after the other, so that the blocks of a wave share both in the L2.
__device__ __forceinline__ void tile_at(const MatmulArgs& a, int64_t t, int& m, int& n) {
    constexpr int kBand = 16;
    const int64_t per_band = static_cast<int64_t>(kBand) * a.n_tiles;
    const int band = static_cast<int>(t / per_band);
    const int rows = min(kBand, a.m_tiles - band * kBand);
    const int rest = static_cast<int>(t - band * per_band);
    n = rest / rows;
    m = band * kBand + rest - n * rows;
}

// Threads: the warps that add up, the issuer's, the loaders', and for two groups of adders a
// group's rest, since registers are handed over by groups of four warps.
constexpr int wide_threads(int n, bool tma) { return n == 256 ? 384 : n + 32 + (tma ? 32 : kLoaders); }
constexpr int thin_threads(bool tma) { return 160 + (tma ? 32 : kLoaders); }

template <int DT, int BN, bool TMA>
__global__ void __launch_bounds__(wide_threads(BN, TMA), 1)
    matmul_wide(const MatmulArgs a, const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap) {
    constexpr int STAGES = wide_stages(BN), BUFFERS = wide_buffers(BN);
    constexpr uint32_t kStage = kTileBytes + BN * kTileK;
    extern __shared__ char dynamic[];
    __shared__ Bars<STAGES, BUFFERS> bars;
    const uint32_t tiles = (smem_u32(dynamic) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kIssuer = BN / 32, kProducer = kIssuer + 1;
    if (warp == kIssuer) tmem_alloc(smem_u32(&bars.tmem), 512);
    if (threadIdx.x == 0) bars.init(TMA ? 1 : kLoaders, BN / 32);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = bars.tmem;
    griddep_wait();
    const int64_t all = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    // of two groups of adders the 384 threads have 168 registers at first: the 8 warps that add
    // up take 232, the other 4 keep 40
    if (warp >= kIssuer) {
        if constexpr (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp >= kProducer) {
            if (TMA ? warp == kProducer && lane == 0 : true) {
                Ring<STAGES> s;
                int64_t issued = 0;
                bool ok = true;
                for (int64_t t = blockIdx.x; ok && t < all; t += gridDim.x) {
                    int m, n;
                    tile_at(a, t, m, n);
                    for (int kb = 0; kb < a.kblocks; ++kb) {
                        if (!(ok = mbar_wait_bounded(smem_u32(&bars.empty[s.at]), s.phase ^ 1u, a.err))) break;
                        const uint32_t dst = tiles + s.at * kStage, full = smem_u32(&bars.full[s.at]);
                        if constexpr (TMA) {
                            mbar_arrive_expect_tx(full, kStage);
                            tile_g2s(dst, &amap, kb * kTileK, m * 128, full);
                            tile_g2s(dst + kTileBytes, &bmap, kb * kTileK, n * BN, full);
                        } else {
                            const int thread = threadIdx.x - kProducer * 32;
                            load_tile<128>(dst, a.a, a.lda, static_cast<int64_t>(m) * 128, a.M, kb * kTileK, a.K, thread);
                            load_tile<BN>(dst + kTileBytes, a.b, a.ldb, static_cast<int64_t>(n) * BN, a.N, kb * kTileK, a.K, thread);
                            fence_proxy_async_smem();
                            mbar_arrive(full);
                        }
                        ++issued;
                        s.next();
                    }
                }
                if (TMA && !ok) drain_tiles(bars, issued, a.err);
            }
            __syncwarp();
        } else if (warp == kIssuer) {
            if (lane == 0) {
                const int64_t mine = all > blockIdx.x ? (all - blockIdx.x - 1) / gridDim.x + 1 : 0;
                issue<STAGES, BUFFERS, BN>(bars, tiles, tmem, mine * a.kblocks, a.err);
            }
            __syncwarp();
        }
    } else {
        if constexpr (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int half = warp >> 2;  // of the tile's columns, 128 each
        const uint32_t mine = tmem + (static_cast<uint32_t>(warp & 3) << 21) + half * 128;
        Ring<BUFFERS> b;
        bool ok = true;
        for (int64_t t = blockIdx.x; t < all; t += gridDim.x) {
            __syncwarp();
            if (!ok) break;  // in all lanes
            int m, n;
            tile_at(a, t, m, n);
            const int64_t row = static_cast<int64_t>(m) * 128 + (warp & 3) * 32 + lane;
            const int col = n * BN + half * 128;
            const bool live = row < a.M && col < a.N;
            const float* sa = a.sa + (live ? row * a.ldsa : 0);
            const float* sb = a.sb + (live ? (col >> 7) * a.ldsb : 0);
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0ull;
            float fa = live ? sa[0] : 0.f, fb = live ? sb[0] : 0.f;
            for (int kb = 0; kb < a.kblocks; ++kb) {
                const float f = fa * fb;
                if (live && kb + 1 < a.kblocks) {
                    if (!a.per_row) fa = sa[kb + 1];
                    fb = sb[kb + 1];
                }
                ok = mbar_wait_bounded(smem_u32(&bars.done[b.at]), b.phase, a.err);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tmem_fence_after();
                const uint64_t f2 = f2_pack(f, f);
                add_up<128>(mine + b.at * BN, acc, smem_u32(&bars.taken[b.at]), [&](int) { return f2; });
                b.next();
            }
            __syncwarp();
            if (!ok || !live) continue;
            constexpr int EB = Elem<DT>::kBytes, V = Elem<DT>::kVec;
            char* out = static_cast<char*>(a.y) + (row * a.ldy + col) * EB;
#pragma unroll
            for (int c = 0; c < 128; c += V) {
                float v[V];
#pragma unroll
                for (int i = 0; i < V; i += 2) f2_unpack(acc[(c + i) / 2], v[i], v[i + 1]);
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
    griddep_launch_dependents();
    tmem_fence_before();
    __syncthreads();
    if (warp == kIssuer) tmem_free(tmem, 512);
}

// Few rows of a: 128 rows of b are the accumulator's lanes, NT rows of a its columns. The
// blocks of a cluster take a part of K each; their sums meet in shared memory and are
// added in the blocks' order, so that the result does not depend on who was first.
template <int DT, int NT, bool TMA>
__global__ void __launch_bounds__(thin_threads(TMA), 1)
    matmul_thin(const MatmulArgs a, const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap) {
    constexpr int STAGES = thin_stages(NT), BUFFERS = kThinBuffers;
    constexpr uint32_t kStage = kTileBytes + NT * kTileK;
    extern __shared__ char dynamic[];
    __shared__ Bars<STAGES, BUFFERS> bars;
    __shared__ alignas(16) float factors[2][NT];
    const uint32_t base = smem_u32(dynamic), tiles = (base + 1023u) & ~1023u;
    float* sums = reinterpret_cast<float*>(dynamic + (tiles - base));  // [NT][128], where the tiles were
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kIssuer = 4, kProducer = 5;
    if (warp == kIssuer) tmem_alloc(smem_u32(&bars.tmem), thin_columns(NT));
    if (threadIdx.x == 0) bars.init(TMA ? 1 : kLoaders, 4);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = bars.tmem;
    griddep_wait();
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
        if (!TMA || lane == 0) {
            Ring<STAGES> s;
            int64_t issued = 0;
            for (int kb = from; kb < to; ++kb) {
                if (!(ok = mbar_wait_bounded(smem_u32(&bars.empty[s.at]), s.phase ^ 1u, a.err))) break;
                const uint32_t dst = tiles + s.at * kStage, full = smem_u32(&bars.full[s.at]);
                if constexpr (TMA) {
                    mbar_arrive_expect_tx(full, kStage);
                    tile_g2s(dst, &bmap, kb * kTileK, n * 128, full);
                    tile_g2s(dst + kTileBytes, &amap, kb * kTileK, m * NT, full);
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
        }
        __syncwarp();
    } else if (warp == kIssuer) {
        if (lane == 0) issue<STAGES, BUFFERS, NT>(bars, tiles, tmem, to - from, a.err);
        __syncwarp();
    } else {
        const uint32_t mine = tmem + (static_cast<uint32_t>(warp) << 21);
        // thread j has the scales of row j
        const bool has = static_cast<int>(threadIdx.x) < rows;
        const float* sa = a.sa + (has ? (t0 + threadIdx.x) * a.ldsa : 0);
        const float* sb = a.sb + n * a.ldsb;
        float fa = has ? sa[a.per_row ? 0 : from] : 0.f, fb = sb[from];
        uint64_t acc[NT / 2];
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) acc[i] = 0ull;
        Ring<BUFFERS> b;
        for (int kb = from; kb < to; ++kb) {
            float* f = factors[kb & 1];
            if (static_cast<int>(threadIdx.x) < NT) f[threadIdx.x] = fa * fb;
            if (kb + 1 < to) {
                if (has && !a.per_row) fa = sa[kb + 1];
                fb = sb[kb + 1];
            }
            named_barrier_sync(1, 128);
            ok = mbar_wait_bounded(smem_u32(&bars.done[b.at]), b.phase, a.err) && ok;
            ok = __all_sync(0xffffffffu, ok);
            // (a wait that gave up: the others go on meeting at the barrier)
            if (ok) {
                tmem_fence_after();
                add_up<NT>(mine + b.at * NT, acc, smem_u32(&bars.taken[b.at]),
                           [&](int c) { return *reinterpret_cast<const uint64_t*>(f + c); });
            }
            b.next();
        }
        const float bias = a.bias && col < a.N ? Elem<DT>::ld(a.bias, col) : 0.f;
        if (split == 1) {
            if (ok && col < a.N) {
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    float v0, v1;
                    f2_unpack(acc[j / 2], v0, v1);
                    if (j < rows) Elem<DT>::st(static_cast<char*>(a.y) + ((t0 + j) * a.ldy + col) * EB, 0, v0 + bias);
                    if (j + 1 < rows) Elem<DT>::st(static_cast<char*>(a.y) + ((t0 + j + 1) * a.ldy + col) * EB, 0, v1 + bias);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NT; j += 2)
                f2_unpack(acc[j / 2], sums[j * 128 + threadIdx.x], sums[(j + 1) * 128 + threadIdx.x]);
        }
    }
    griddep_launch_dependents();
    __syncwarp();
    if (split > 1) {
        cluster_sync();
        if (warp < 4 && ok && col < a.N) {
            const float bias = a.bias ? Elem<DT>::ld(a.bias, col) : 0.f;
            const uint32_t at = smem_u32(sums) + threadIdx.x * 4;
            for (int j = rank; j < rows; j += split) {
                float v = 0.f;
                for (int r = 0; r < split; ++r) v += dsmem_ld_f32(dsmem_map(at + j * 512, r));
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
    if (p.wide) {
        if constexpr (TMA)
            if (p.n == 256) return reinterpret_cast<const void*>(&matmul_wide<DT, 256, TMA>);
        return p.n == 128 ? reinterpret_cast<const void*>(&matmul_wide<DT, 128, TMA>) : nullptr;
    }
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
    const int stages = p.wide ? wide_stages(p.n) : thin_stages(p.n);
    p.threads = p.wide ? wide_threads(p.n, p.tma) : thin_threads(p.tma);
    p.smem = 1024 + static_cast<size_t>(stages) * (kTileBytes + p.n * kTileK);
}

}  // namespace rmsnorm
