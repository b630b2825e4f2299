// matmul.cu -- products of e4m3 codes with scales: y = (a sa) (b sb)^T + bias.
//
// a is [M, K] with a scale per row and 128 columns (or per row), b [N, K] with one per
// block of 128 x 128. Over one block of 128 columns both scales of an element of y are
// constants, so
//     y[m, n] = sum over blocks j of sa[m, j] * sb[n / 128, j] * (a_j b_j^T)[m, n].
// The inner products of a block, 128 products of codes, are summed by the tensor cores in
// fp32; the sum over blocks is taken in fp32 registers, by one multiply-add per element and
// block.
//
// Three kernels. matmul_pair: pairs of blocks on tiles of 256 x 256, a thread to a row of the
// accumulator. matmul_wide: single blocks on tiles of 128 x 128. matmul_thin, for few rows
// of a: the operands change places, a tile is 128 rows of b and 16 to 64 of a. Where tiles are
// few the blocks of a cluster share a tile's K. In all of them one warp keeps a ring of tiles full
// by TMA, one issues the matrix instructions into one of several accumulators in tensor
// memory, and warps of four add finished ones up meanwhile. Rows off 16 bytes, which TMA does not
// take, are copied as they lie by eight warps, which shift them into the tiles.
//
// Measured on GB300 (device copy 6.79 TB/s; bf16 products of the library 1.94 PFLOP/s, 1.73 under
// the power limit): 16384 x 8192 x 8192 into bf16 830-850 us (2.6 PFLOP/s at 1350 W, the power
// limit; the tensor cores are busy for half of the time, and the sums, 128 multiply-adds a
// thread and block, bound the rest), 2048 x 4096 x 5120 into fp32 with a bias 41 us (128 tiles
// are two turns of 76 pairs), 512 x 4096 x 4096 12.5 us, 64 x 8192 x 8192 17.3 us and 8 x 6144 x
// 4096 8 us (the weight's bytes in 11 and 3.4 us of it, at 6 to 7 TB/s; the rest is the start
// of a ring, 1.2 us, and the meeting of a cluster's sums, 1.5 to 2.5), 1001 x 5120 x 4099, rows off 16
// bytes, 108 us.
#include "octet.cuh"
#include "serving.h"
#include "tcgen05.cuh"

namespace rmsnorm {
namespace {

constexpr int kTileBytes = 128 * kTileK;  // 128 rows

constexpr int kPairStages = 6;
// Two blocks to an SM, where rows need no raw place.
constexpr int thin_blocks(bool tma) { return tma ? 2 : 1; }
constexpr int thin_stages(int n, bool tma) { return tma && n < 32 ? 5 : 4; }
// Accumulators in tensor memory that are under way.
constexpr int kWideBuffers = 4, kPairBuffers = 2;
constexpr int kThinBuffers = 4;
constexpr int thin_columns(int n) { return kThinBuffers * n; }

// 32 bytes, of which the 16 from byte `sh` on come back.
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, uint32_t sh) {
    uint32_t s[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (sh & 8u) {
#pragma unroll
        for (int i = 0; i < 6; ++i) s[i] = s[i + 2];
    }
    if (sh & 4u) {
#pragma unroll
        for (int i = 0; i < 5; ++i) s[i] = s[i + 1];
    }
    const uint32_t bits = 8u * (sh & 3u);
    return make_uint4(__funnelshift_r(s[0], s[1], bits), __funnelshift_r(s[1], s[2], bits), __funnelshift_r(s[2], s[3], bits),
                      __funnelshift_r(s[3], s[4], bits));
}

// The first n of 16 codes, the others 0.
__device__ __forceinline__ uint4 first_codes(uint4 v, int n) {
    const auto part = [&](uint32_t w, int at) { return n >= at + 4 ? w : n <= at ? 0u : w & ((1u << (8 * (n - at))) - 1u); };
    return make_uint4(part(v.x, 0), part(v.y, 4), part(v.z, 8), part(v.w, 12));
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
// and one for the instructions under way when a wait has given up; and whether one of the warps that
// add up has, for the other blocks of a cluster.
template <int STAGES, int BUFFERS> struct Bars {
    uint64_t full[STAGES], empty[STAGES], done[BUFFERS], taken[BUFFERS], drain;
    uint32_t tmem, gave_up;
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
        gave_up = 0;
        fence_mbar_init();
    }
    // Before the cluster's sums meet: whether this warp's are whole. In debug builds those of a
    // chosen block's first warp never are.
    __device__ __forceinline__ bool whole(const MatmulArgs& a, int rank, int warp, bool ok) {
        if (kDebugReads && rank == a.give_up && warp == 0) {
            if ((threadIdx.x & 31) == 0) atomicOr(a.err, kDevErrWaitTimeout);
            ok = false;
        }
        if (!ok && (threadIdx.x & 31) == 0) gave_up = 1;
        return ok;
    }
};

// The warp that issues matrix instructions: `blocks` blocks of K through the ring (a stage has a tile
// of 128 rows and one of Y) into the accumulators in turn. PAIR: for both blocks of a cluster, 256
// rows by 256. The loop is the whole warp's, see elect_lane (16384 x 8192 x 8192 1110 us with a
// loop of one thread).
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

// Rows off 16 bytes. A row of a block of K lies in 9 words of 16 bytes at most. Each of kLoaders / 32
// warps copies its rows' words as they are into one of three places (cp.async, three blocks ahead;
// words without a code of the row are not read and become zeros), and then moves the rows' 16-byte
// pieces, shifted from two words, to their swizzled places in the tile. No warp waits for
// another's rows. Bound by the L1's pipeline: a row of 144 bytes touches two lines (without the copies
// 83 us, without the shifts 68, without both 33), and a tile goes through shared memory three times.
// 1001 x 5120 x 4099 108 us; 574 with single loads and the shift in between, 126 with all loaders'
// rows behind one barrier, 129 with twice the loaders in two groups that take the blocks in turn, 207 with a
// bulk copy of each row.
constexpr int kLoaders = 256, kLoaderWarps = kLoaders / 32;
constexpr int kRawWords = kTileK / 16 + 1, kRawAhead = 3;
constexpr int kRawRow = 16 * kRawWords;

struct RawSide {
    const uint8_t* base;
    int64_t ld, row0, rows;
};

// A lane's part of R rows of a warp (the first is row0 of the matrix): its words in the first block
// of K, and from how many codes of a block on they hold one; and the pieces that it shifts.
template <int R> struct RawRows {
    static constexpr int kAll = R * kRawWords, kMine = (kAll + 31) / 32;
    static constexpr int kPieces = R * 8, kShifts = (kPieces + 31) / 32;
    const uint8_t* src[kMine];
    int from[kMine];
    uint32_t sh[kShifts];  // a piece's row's offset from a 16-byte boundary: tiles start 16 rows apart at
                           // least, so that it is the same for each, also while the next one is copied
    const uint8_t* any;    // a word that may be named where none is read
    __device__ __forceinline__ void rows(const RawSide& x, int64_t row0, int lane) {
        any = x.base - (reinterpret_cast<uintptr_t>(x.base) & 15);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int at = i * 32 + lane, row = at / kRawWords, word = at - row * kRawWords;
            const bool in = at < kAll && row0 + row < x.rows;
            const uint8_t* p = x.base + (in ? (row0 + row) * x.ld : 0);
            const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
            src[i] = p - off + 16 * word;
            from[i] = in ? 16 * word - off : kTileK;
        }
        const uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x.base)), ld = static_cast<uint32_t>(x.ld);
#pragma unroll
        for (int i = 0; i < kShifts; ++i) sh[i] = (low + static_cast<uint32_t>(row0 + ((i * 32 + lane) >> 3)) * ld) & 15u;
    }
    // Block kb, of which `left` codes are the rows'.
    __device__ __forceinline__ void copy(uint32_t raw, int kb, int left, int lane) const {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            if (kAll % 32 != 0 && i * 32 + lane >= kAll) break;
            const bool some = from[i] < left;
            const uint8_t* p = some ? src[i] + static_cast<int64_t>(kb) * kTileK : any;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(raw + (i * 32 + lane) * 16), "l"(p),
                         "r"(some ? 16 : 0)
                         : "memory");
        }
    }
    // The rows from `raw` into the tile, the first of them its row `first`.
    __device__ __forceinline__ void shift(uint32_t tile, const char* raw, int first, int left, int lane) const {
#pragma unroll
        for (int i = 0; i < kShifts; ++i) {
            const int at = i * 32 + lane, row = at >> 3, c = at & 7;
            if (kPieces % 32 != 0 && at >= kPieces) break;
            const uint4* p = reinterpret_cast<const uint4*>(raw + row * kRawRow + c * 16);
            uint4 v = shifted(p[0], p[1], sh[i]);
            if (left < kTileK) v = first_codes(v, left - 16 * c);
            const uint32_t to = tile + (first + row) * kTileK + ((c ^ ((first + row) & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
        }
    }
};

// The tiles of X rows and of Y by the loaders. at.next(kb): the next block of K and whether there is
// one; at.rows(x, y): its tile's rows on both sides, which change where kb is `from`.
template <int STAGES, int BUFFERS, int X, int Y, class At>
__device__ __forceinline__ void load_tiles(Bars<STAGES, BUFFERS>& bars, uint32_t tiles, char* raw, const MatmulArgs& a, int from,
                                           int thread, At at) {
    constexpr uint32_t kStage = (X + Y) * kTileK;
    constexpr int RX = X / kLoaderWarps, RY = Y / kLoaderWarps, kRaw = (X + Y) * kRawRow;
    const int warp = thread >> 5, lane = thread & 31;
    raw += warp * (RX + RY) * kRawRow;
    At ahead = at;
    RawRows<RX> wx;
    RawRows<RY> wy;
    int slot = 0, to = 0;
    const auto copy = [&] {
        int kb;
        if (ahead.next(kb)) {
            if (kb == from) {
                RawSide x, y;
                ahead.rows(x, y);
                wx.rows(x, x.row0 + warp * RX, lane);
                wy.rows(y, y.row0 + warp * RY, lane);
            }
            const uint32_t dst = smem_u32(raw) + to * kRaw;
            const int left = min(a.K - kb * kTileK, kTileK);
            wx.copy(dst, kb, left, lane);
            wy.copy(dst + RX * kRawRow, kb, left, lane);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        to = to == kRawAhead - 1 ? 0 : to + 1;
    };
    for (int i = 0; i < kRawAhead; ++i) copy();
    Ring<STAGES> s;
    int kb;
    while (at.next(kb)) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRawAhead - 1) : "memory");
        const bool ok = mbar_wait_bounded(smem_u32(bars.empty) + 8 * s.at, s.phase ^ 1u, a.err);
        if (!__all_sync(0xffffffffu, ok)) break;
        __syncwarp();  // the words that the other lanes waited for are there
        const uint32_t dst = tiles + s.at * kStage;
        const int left = a.K - kb * kTileK;
        wx.shift(dst, raw + slot * kRaw, warp * RX, left, lane);
        wy.shift(dst + X * kTileK, raw + slot * kRaw + RX * kRawRow, warp * RY, left, lane);
        fence_proxy_async_smem();
        __syncwarp();  // (and the place is free again)
        if (lane == 0) mbar_arrive(smem_u32(bars.full) + 8 * s.at);
        copy();
        slot = slot == kRawAhead - 1 ? 0 : slot + 1;
        s.next();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// After a wait that gave up: the tiles that are still on their way, `issued` in all.
template <int STAGES, int BUFFERS>
__device__ __forceinline__ void drain_tiles(Bars<STAGES, BUFFERS>& bars, int64_t issued, uint32_t* err) {
    for (int64_t i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
        mbar_wait_bounded(smem_u32(&bars.full[i % STAGES]), static_cast<uint32_t>(i / STAGES & 1), err);
}

// A finished accumulator's columns [0, C) of this thread's row, each times its factor (given for
// four columns), added to acc; `arrive` gives it back as soon as it is in registers. Single multiply-adds: packed pairs
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

// A row's scale times its columns' block's, of the blocks of K one after the other from `from`
// to `to`, loaded a block ahead.
struct Scales {
    const float *sa, *sb;
    float fa, fb;
    bool live, per_row;
    __device__ __forceinline__ Scales(const MatmulArgs& a, int64_t row, int col, int from)
        : live(row < a.M && col < a.N), per_row(a.per_row != 0) {
        sa = a.sa + (live ? row * a.ldsa + (per_row ? 0 : from) : 0);
        sb = a.sb + (live ? (col >> 7) * a.ldsb + from : 0);
        fa = live ? *sa : 0.f;
        fb = live ? *sb : 0.f;
    }
    __device__ __forceinline__ float next(bool more) {
        const float f = fa * fb;
        if (live && more) {
            if (!per_row) fa = *++sa;
            fb = *++sb;
        }
        return f;
    }
};

// 128 sums before the first block of K: the bias of their columns, or 0.
template <int DT>
__device__ __forceinline__ void start_sums(const MatmulArgs& a, int col, bool bias, float (&acc)[128]) {
    constexpr int EB = Elem<DT>::kBytes, V = Elem<DT>::kVec;
#pragma unroll
    for (int i = 0; i < 128; ++i) acc[i] = 0.f;
    if (!bias || !a.bias) return;
    if (a.wide_bias && col + 128 <= a.N) {
#pragma unroll
        for (int c = 0; c < 128; c += V)
            Elem<DT>::unpack(__ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(a.bias) + (col + c) * EB)),
                             *reinterpret_cast<float(*)[V]>(&acc[c]));
    } else {
#pragma unroll
        for (int i = 0; i < 128; ++i)
            if (col + i < a.N) acc[i] = Elem<DT>::ld(a.bias, col + i);
    }
}

// The blocks of K from `from` to `to` of this thread's row and 128 columns (at `mine` in tensor
// memory) added up, with the bias or without; false where a wait gave up (in all lanes).
template <int DT, int BN, int BUFFERS, class Done, class Taken>
__device__ __forceinline__ bool add_blocks(const MatmulArgs& a, uint32_t mine, int64_t row, int col, int from, int to, bool bias,
                                           Ring<BUFFERS>& b, float (&acc)[128], Done&& done, Taken&& taken) {
    Scales scales(a, row, col, from);
    start_sums<DT>(a, col, bias, acc);
    for (int kb = from; kb < to; ++kb) {
        const float f = scales.next(kb + 1 < to);
        const bool ok = mbar_wait_bounded(done(b.at), b.phase, a.err);
        if (!__all_sync(0xffffffffu, ok)) return false;
        tmem_fence_after();
        add_up<128>(mine + b.at * BN, acc, [&] { taken(b.at); }, [&](int) { return make_float4(f, f, f, f); });
        b.next();
    }
    return true;
}

// Places for 64 bytes of a warp's 32 rows, 80 apart: 16-byte pieces of 8 rows touch every bank once.
constexpr int kPieceRow = 80;
struct RowPieces {
    alignas(16) char at[32 * kPieceRow];
};

// A warp's 32 rows (from row0 on, a thread's sums its own row's) of 128 columns (from col on) to y.
// They change places in shared memory, 64 bytes of each row at a time, so that four lanes store
// a row's 64 bytes (a thread storing its own row's pieces touches 32 lines with every
// store: 2048 x 4096 x 5120 into fp32 58 us), or 32 lanes single entries side by side
// where y's rows are off 16 bytes.
template <int DT>
__device__ __forceinline__ void store_rows(const MatmulArgs& a, RowPieces& pieces, int64_t row0, int col, const float (&acc)[128]) {
    constexpr int EB = Elem<DT>::kBytes, V = Elem<DT>::kVec, C = 64 / EB;
    const int lane = threadIdx.x & 31;
    char* const mine = pieces.at + lane * kPieceRow;
    const int rows = static_cast<int>(min(int64_t(32), a.M - row0)), cols = min(128, a.N - col);
    char* const out = static_cast<char*>(a.y) + (row0 * a.ldy + col) * EB;
#pragma unroll
    for (int c = 0; c < 128; c += C) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = acc[c + V * u + i];
            *reinterpret_cast<uint4*>(mine + 16 * u) = Elem<DT>::pack(v);
        }
        __syncwarp();
        if (a.wide_y && c + C <= cols) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * i + (lane >> 2);
                if (r < rows)
                    *reinterpret_cast<uint4*>(out + (r * a.ldy + c) * EB + (lane & 3) * 16) =
                        *reinterpret_cast<const uint4*>(pieces.at + r * kPieceRow + (lane & 3) * 16);
            }
        } else {
            constexpr int R = 32 / C;  // rows at a time
            const int k = lane % C;
            if (c + k < cols) {
#pragma unroll 4
                for (int r = lane / C; r < rows; r += R) {
                    const char* from = pieces.at + r * kPieceRow + k * EB;
                    char* to = out + (r * a.ldy + c + k) * EB;
                    if constexpr (EB == 4) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(from);
                    else *reinterpret_cast<uint16_t*>(to) = *reinterpret_cast<const uint16_t*>(from);
                }
            }
        }
        __syncwarp();
    }
}

// The blocks of K of a cluster's block.
struct Share {
    int from, to;
    __device__ __forceinline__ Share(const MatmulArgs& a, int rank, int split)
        : from(static_cast<int>(static_cast<int64_t>(a.kblocks) * rank / split)),
          to(static_cast<int>(static_cast<int64_t>(a.kblocks) * (rank + 1) / split)) {}
};

// The cluster's sums [rows][PITCH], at one place in its blocks' shared memory, added in the blocks'
// order and stored, four warps of a block to every split-th four rows: row r is row0 + r of y,
// its 128 columns are those from col0 on, four to a lane. Four rows and four blocks at a time,
// whose loads are under way together. Nothing is stored where a block's `gave_up` is set: its sums
// lack blocks of K.
template <int DT, int PITCH>
__device__ __forceinline__ void store_cluster(const MatmulArgs& a, uint32_t gave_up, uint32_t sums, int64_t row0, int rows,
                                              int col0, int rank, int split, int warp) {
    constexpr int EB = Elem<DT>::kBytes, B = 4;
    const int lane = threadIdx.x & 31, col = col0 + 4 * lane;
    const uint32_t lacking = lane < split ? dsmem_ld_u32(dsmem_map(gave_up, lane)) : 0u;
    float bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = a.bias && col + i < a.N ? Elem<DT>::ld(a.bias, col + i) : 0.f;
    const int step = 4 * split;
    for (int first = rank * 4 + warp; first < rows; first += B * step) {
        float v[B][4];
#pragma unroll
        for (int i = 0; i < B; ++i) v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
#pragma unroll 1
        for (int k0 = 0; k0 < split; k0 += 4) {
            float4 part[B][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t from = dsmem_map(sums, min(k0 + k, split - 1));
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    part[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k0 + k < split && first + i * step < rows)
                        part[i][k] = dsmem_ld_f4(from + ((first + i * step) * PITCH + 4 * lane) * 4);
                }
            }
#pragma unroll
            for (int i = 0; i < B; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[i][0] += part[i][k].x;
                    v[i][1] += part[i][k].y;
                    v[i][2] += part[i][k].z;
                    v[i][3] += part[i][k].w;
                }
        }
        if (__any_sync(0xffffffffu, lacking != 0u)) return;
#pragma unroll
        for (int i = 0; i < B; ++i) {
            if (first + i * step >= rows) break;
#pragma unroll
            for (int c = 0; c < 4; ++c) v[i][c] += bias[c];
            char* out = static_cast<char*>(a.y) + ((row0 + first + i * step) * a.ldy + col) * EB;
            if (a.wide_y && col + 4 <= a.N) {
                if constexpr (EB == 4) *reinterpret_cast<float4*>(out) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
                else
                    *reinterpret_cast<uint2*>(out) =
                        make_uint2(Elem<DT>::pack2(v[i][0], v[i][1]), Elem<DT>::pack2(v[i][2], v[i][3]));
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (col + c < a.N) Elem<DT>::st(out, c, v[i][c]);
            }
        }
    }
}

// Threads: the warps that add up, the issuer's, and the one that loads by TMA; or, where loaders
// shift rows, and in pairs, groups of four warps throughout, between which registers are handed over.
constexpr int tile_threads(bool tma) { return tma ? 192 : 256 + kLoaders; }
constexpr int kPairThreads = 384;
// Registers of a thread that adds up, of the issuer's group and of a loader. A group that asks for
// more than all have at launch would wait for ever.
constexpr int kAddRegs = 232, kIssueRegs = 40, kLoadRegs = 120;
constexpr int launch_regs(int threads) { return 65536 / threads / 8 * 8; }
static_assert(kAddRegs + kIssueRegs + kLoaders / 128 * kLoadRegs <= tile_threads(false) / 128 * launch_regs(tile_threads(false)),
              "registers of loaders' blocks");
static_assert(2 * kAddRegs + kIssueRegs <= kPairThreads / 128 * launch_regs(kPairThreads), "registers of pairs");
template <int REGS> __device__ __forceinline__ void take_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS> __device__ __forceinline__ void give_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
// Stages of the tiles, and behind them the raw rows of the loaders.
constexpr int wide_stages(bool tma) { return tma ? 6 : 3; }
constexpr size_t raw_bytes(int rows, bool tma) { return tma ? 0 : static_cast<size_t>(kRawAhead) * rows * kRawRow; }

constexpr int kWidePitch = 132;  // of a row of sums: 16-byte pieces of 8 rows touch every bank once

// The blocks of K of a persistent block's tiles, for load_tiles.
struct WideBlocks {
    const MatmulArgs& a;
    int64_t turn, step, all;
    Share share;
    int kb;
    __device__ __forceinline__ bool next(int& now) {
        if (kb == share.to) {
            kb = share.from;
            turn += step;
        }
        now = kb++;
        return turn < all;
    }
    __device__ __forceinline__ void rows(RawSide& x, RawSide& y) const {
        int m, n;
        tile_at(a, turn, m, n);
        x = {a.a, a.lda, static_cast<int64_t>(m) * 128, a.M};
        y = {a.b, a.ldb, static_cast<int64_t>(n) * 128, a.N};
    }
};
// Those of one tile.
struct ThinBlocks {
    RawSide x, y;
    int kb, to;
    __device__ __forceinline__ bool next(int& now) {
        now = kb++;
        return now < to;
    }
    __device__ __forceinline__ void rows(RawSide& xs, RawSide& ys) const {
        xs = x;
        ys = y;
    }
};

// One block to a tile, persistent; or, where tiles are few, the blocks of a cluster to a tile, a
// part of K each.
template <int DT, bool TMA>
__global__ void __launch_bounds__(tile_threads(TMA), 1)
    matmul_wide(const MatmulArgs a, const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap) {
    constexpr int STAGES = wide_stages(TMA), BUFFERS = kWideBuffers;
    constexpr uint32_t kStage = 2 * kTileBytes;
    extern __shared__ char dynamic[];
    __shared__ Bars<STAGES, BUFFERS> bars;
    __shared__ RowPieces pieces[4];
    const uint32_t base = smem_u32(dynamic), tiles = (base + 1023u) & ~1023u;
    char* const first_tile = dynamic + (tiles - base);
    float* const sums = reinterpret_cast<float*>(first_tile);  // [128][kWidePitch], where the tiles were
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform to the compiler
    if (warp == 4) tmem_alloc(smem_u32(&bars.tmem), 512);
    if (threadIdx.x == 0) bars.init(TMA ? 1 : kLoaderWarps, 4);
    if (TMA && threadIdx.x == 160) {
        prefetch_map(&amap);
        prefetch_map(&bmap);
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = bars.tmem;
    griddep_wait();
    const int split = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    const int64_t all = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    const int64_t first = blockIdx.x / split, step = gridDim.x / split;
    const Share share(a, rank, split);
    if (warp >= 4) {
        if constexpr (!TMA) {
            if (warp < 8) give_registers<kIssueRegs>();
            else give_registers<kLoadRegs>();
        }
        if (warp == 4) {
            const int64_t mine = all > first ? (all - first - 1) / step + 1 : 0;
            issue<STAGES, BUFFERS, 128, false>(bars, tiles, tmem, mine * (share.to - share.from), a.err);
        } else if (TMA) {
            Ring<STAGES> s;
            int64_t issued = 0;
            bool ok = true;
            for (int64_t turn = first; ok && turn < all; turn += step) {
                int m, n;
                tile_at(a, turn, m, n);
                for (int kb = share.from; kb < share.to; ++kb) {
                    ok = mbar_wait_bounded(smem_u32(bars.empty) + 8 * s.at, s.phase ^ 1u, a.err);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    if (elect_lane()) {
                        const uint32_t dst = tiles + s.at * kStage, full = smem_u32(bars.full) + 8 * s.at;
                        mbar_arrive_expect_tx(full, kStage);
                        tile_g2s(dst, &amap, kb * kTileK, m * 128, full);
                        tile_g2s(dst + kTileBytes, &bmap, kb * kTileK, n * 128, full);
                    }
                    __syncwarp();
                    ++issued;
                    s.next();
                }
            }
            if (!ok) drain_tiles(bars, issued, a.err);
        } else if (warp >= 8) {
            const int thread = threadIdx.x - 256;
            load_tiles<STAGES, BUFFERS, 128, 128>(bars, tiles, first_tile + STAGES * kStage, a, share.from, thread,
                                                  WideBlocks{a, first, step, all, share, share.from});
        }
        __syncwarp();
        if (split > 1) {
            cluster_sync();
            cluster_sync();
        }
    } else {
        if constexpr (!TMA) take_registers<kAddRegs>();
        const uint32_t mine = tmem + (static_cast<uint32_t>(warp) << 21);
        Ring<BUFFERS> b;
        bool ok = true;
        int m = 0, n = 0;
        for (int64_t turn = first; ok && turn < all; turn += step) {
            tile_at(a, turn, m, n);
            const int64_t row = static_cast<int64_t>(m) * 128 + threadIdx.x;
            float acc[128];
            ok = add_blocks<DT, 128, BUFFERS>(a, mine, row, n * 128, share.from, share.to, split == 1, b, acc,
                                          [&](int i) { return smem_u32(bars.done) + 8 * i; },
                                          [&](int i) { mbar_arrive(smem_u32(bars.taken) + 8 * i); });
            if (split > 1) {
#pragma unroll
                for (int i = 0; i < 128; i += 4)
                    *reinterpret_cast<float4*>(sums + threadIdx.x * kWidePitch + i) =
                        make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
            } else if (ok) {
                store_rows<DT>(a, pieces[warp], row - (threadIdx.x & 31), n * 128, acc);
            }
            __syncwarp();
        }
        if (split > 1) {
            ok = bars.whole(a, rank, warp, ok);
            __syncwarp();
            cluster_sync();
            const int64_t row0 = static_cast<int64_t>(m) * 128;
            const int rows = static_cast<int>(min(int64_t(128), a.M - row0));
            if (ok) store_cluster<DT, kWidePitch>(a, smem_u32(&bars.gave_up), smem_u32(sums), row0, rows, n * 128, rank, split, warp);
            __syncwarp();
            cluster_sync();
        }
    }
    griddep_launch_dependents();
    tmem_fence_before();
    __syncthreads();
    if (warp == 4) tmem_free(tmem, 512);
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
    __shared__ RowPieces pieces[8];
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
    if (warp >= kIssuer) {
        give_registers<kIssueRegs>();
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
        take_registers<kAddRegs>();
        const int half = warp >> 2;  // of the tile's columns
        const uint32_t mine = tmem + (static_cast<uint32_t>(warp & 3) << 21) + half * 128;
        Ring<BUFFERS> b;
        bool ok = true;
        for (int64_t turn = first; ok && turn < all; turn += step) {
            int m, n;
            tile_at(a, turn, m, n);
            const int64_t row = static_cast<int64_t>(m) * 256 + rank * 128 + (threadIdx.x & 127);
            const int col = n * 256 + half * 128;
            float acc[128];
            ok = add_blocks<DT, 256, BUFFERS>(a, mine, row, col, 0, a.kblocks, true, b, acc,
                                              [&](int i) { return smem_u32(bars.done) + 8 * i; },
                                              [&](int i) { mbar_arrive_cluster(dsmem_map(smem_u32(bars.taken) + 8 * i, 0)); });
            if (ok && col < a.N) store_rows<DT>(a, pieces[warp], row - (threadIdx.x & 31), col, acc);
            __syncwarp();
        }
    }
    griddep_launch_dependents();
    tmem_fence_before();
    __syncwarp();
    cluster_sync();  // no block leaves before the other's instructions and arrivals
    if (warp == kIssuer) tmem_free_pair(tmem, 512);
}

// Blocks of K whose factors lie in shared memory at a time.
constexpr int kFactorBlocks = 16;

// Few rows of a: 128 rows of b are the accumulator's lanes, NT rows of a its columns. The
// blocks of a cluster take a part of K each; their sums meet in shared memory and are
// added in the blocks' order, so that the result does not depend on who was first.
template <int DT, int NT, bool TMA>
__global__ void __launch_bounds__(tile_threads(TMA), thin_blocks(TMA))
    matmul_thin(const MatmulArgs a, const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap) {
    constexpr int STAGES = thin_stages(NT, TMA), BUFFERS = kThinBuffers;
    constexpr uint32_t kStage = kTileBytes + NT * kTileK;
    extern __shared__ char dynamic[];
    __shared__ Bars<STAGES, BUFFERS> bars;
    __shared__ alignas(16) float factors[2][kFactorBlocks][NT + 4];
    const uint32_t base = smem_u32(dynamic), tiles = (base + 1023u) & ~1023u;
    char* const first_tile = dynamic + (tiles - base);
    float* const sums = reinterpret_cast<float*>(first_tile);  // [NT][128], where the tiles were
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform to the compiler
    constexpr int kIssuer = 4;
    if (warp == kIssuer) tmem_alloc(smem_u32(&bars.tmem), thin_columns(NT));
    if (threadIdx.x == 0) bars.init(TMA ? 1 : kLoaderWarps, 4);
    if (TMA && threadIdx.x == 160) {
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
    const Share share(a, rank, split);
    const int from = share.from, to = share.to;
    constexpr int EB = Elem<DT>::kBytes;
    const int col = n * 128 + threadIdx.x;  // of y, for the threads that add up
    const int rows = static_cast<int>(min(static_cast<int64_t>(NT), a.M - t0));
    bool ok = true;
    if (warp >= 4) {
        if constexpr (!TMA) {
            if (warp < 8) give_registers<kIssueRegs>();
            else give_registers<kLoadRegs>();
        }
        if (warp == kIssuer) {
            issue<STAGES, BUFFERS, NT, false>(bars, tiles, tmem, to - from, a.err);
        } else if (TMA) {
            Ring<STAGES> s;
            int64_t issued = 0;
            for (int kb = from; kb < to; ++kb) {
                ok = mbar_wait_bounded(smem_u32(bars.empty) + 8 * s.at, s.phase ^ 1u, a.err);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                if (elect_lane()) {
                    const uint32_t dst = tiles + s.at * kStage, full = smem_u32(bars.full) + 8 * s.at;
                    mbar_arrive_expect_tx(full, kStage);
                    tile_g2s(dst, &bmap, kb * kTileK, n * 128, full);
                    tile_g2s(dst + kTileBytes, &amap, kb * kTileK, m * NT, full);
                }
                __syncwarp();
                ++issued;
                s.next();
            }
            if (!ok) drain_tiles(bars, issued, a.err);
        } else if (warp >= 8) {
            const int thread = threadIdx.x - 256;
            const RawSide x = {a.b, a.ldb, static_cast<int64_t>(n) * 128, a.N}, y = {a.a, a.lda, t0, a.M};
            load_tiles<STAGES, BUFFERS, 128, NT>(bars, tiles, first_tile + STAGES * kStage, a, from, thread,
                                                 ThinBlocks{x, y, from, to});
        }
        __syncwarp();
        if (split > 1) {
            cluster_sync();
            cluster_sync();
        }
    } else {
        if constexpr (!TMA) take_registers<kAddRegs>();
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
                ok = ok && mbar_wait_bounded(smem_u32(bars.done) + 8 * b.at, b.phase, a.err);
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
        if (split == 1) {
            const float bias = a.bias && col < a.N ? Elem<DT>::ld(a.bias, col) : 0.f;
            if (ok && col < a.N) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (j < rows) Elem<DT>::st(static_cast<char*>(a.y) + ((t0 + j) * a.ldy + col) * EB, 0, acc[j] + bias);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NT; ++j) sums[j * 128 + threadIdx.x] = acc[j];
            ok = bars.whole(a, rank, warp, ok);
            __syncwarp();
            cluster_sync();
            if (ok) store_cluster<DT, 128>(a, smem_u32(&bars.gave_up), smem_u32(sums), t0, rows, n * 128, rank, split, warp);
            __syncwarp();
            cluster_sync();
        }
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
    const int rows = 128 + (thin ? p.n : 128);
    const int stages = thin ? thin_stages(p.n, p.tma) : p.how == kMatmulWide ? wide_stages(p.tma) : kPairStages;
    p.threads = p.how == kMatmulPair ? kPairThreads : tile_threads(p.tma);
    p.smem = 1024 + static_cast<size_t>(stages) * rows * kTileK + raw_bytes(rows, p.tma);
}

}  // namespace rmsnorm
