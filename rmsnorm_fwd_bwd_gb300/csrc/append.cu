// append.cu -- RMSNorm and rotation of query and key heads, and keys and values written to the
// rows ("slots") of a paged cache, in one launch.
//
// Queries and keys are those of rope.cu: z = x * r * g, and the first R entries turned by the
// token's position. A token's keys and values go to slot s of their caches, row s %
// page_size of page s / page_size; a negative slot stores nothing. A cache holds the rows in
// their own type (values are copied bit by bit), or as e4m3 codes with a scale per head row:
// scale = max(max|z| / 448, 2^-126), code = z / scale rounded to nearest-even; r is left out
// of z until the scale is known and cancels between the two, as in quant.cu.
//
// A group of lanes takes up to a few heads of one kind of one token, as rope.cu's forwards do,
// and writes whole head rows, so that a page's end, or pages in any order, cost nothing.
// Blocks of one kind: with a token's heads of all kinds in a block (and the slot read before the
// heads) the largest case took 176 us.
//
// Bound by HBM, and by instructions where the codes and short rows need them. Measured on GB300 (a
// device copy moves 6.79 TB/s): 32768 tokens x (32 + 2 x 8) heads x 128 bf16, half rotated, into
// an 8-bit cache 134 us (5.5 TB/s), 16384 x (16 + 2 x 4) x 256 fp16 67 us (6.0), 16384 x (32 + 2 x 8) x 128
// bf16 67 us (6.0), 8191 x (28 + 2 x 4) x 80 bf16, a padded batch, 24 us (3.9: five of a group's eight
// lanes have entries), 64 x (32 + 2 x 8) x 128 2.8 us in a graph; partners through shared memory (24 of 128 entries
// rotated) 16384 x 48 heads 100 us (3.7), entry by entry 8192 x 48 x 90 80 us (1.6; 92 with
// a head's loads when its turn comes).
#include "launch.h"
#include "quant.cuh"
#include "rope.cuh"
#include "serving.h"

namespace rmsnorm {
namespace {

// The heads that a group of lanes takes, and where they go. A block's groups take heads of one
// kind (queries, keys or values, in this order of the blocks): what that kind does without is
// skipped by the whole block, and its description is read from the arguments at a known place.
struct Work {
    AppendSet set;
    int kind;
    int64_t token;
    int from, n;       // heads from `from` on, of which there are n
    int stored;        // heads that are stored: n, or none where the token has no slot
    char* out;         // row of head `from`
    int64_t step;      // bytes between heads
    float* scales;     // of head `from`, or null
    __device__ __forceinline__ bool rotate() const { return kind < 2; }
};

__device__ __forceinline__ Work work_of(const AppendArgs& a, int lanes) {
    Work w;
    w.kind = blockIdx.x >= static_cast<unsigned>(a.first[2]) ? 2 : blockIdx.x >= static_cast<unsigned>(a.first[1]) ? 1 : 0;
    w.set = w.kind == 0 ? a.sets[0] : w.kind == 1 ? a.sets[1] : a.sets[2];
    const int first = w.kind == 0 ? 0 : w.kind == 1 ? a.first[1] : a.first[2];
    const int64_t item = static_cast<int64_t>(blockIdx.x - first) * (blockDim.x / lanes) + threadIdx.x / lanes;
    const int nchunk = (w.set.heads + a.chunk - 1) / a.chunk;
    const bool live = item < a.T * nchunk;
    int chunk;
    w.token = split_item(live ? item : 0, nchunk, chunk);
    w.from = chunk * a.chunk;
    w.n = live ? min(a.chunk, w.set.heads - w.from) : 0;
    return w;
}

// Where they go. Apart from work_of, so that the slot is read while the heads are under way. One
// thread of a group reports a slot behind the cache's last.
template <int DT> __device__ __forceinline__ void place(const AppendArgs& a, Work& w, bool reports) {
    const AppendSet& s = w.set;
    w.scales = nullptr;
    w.stored = w.n;
    int64_t page = 0, row = w.token;
    if (w.kind > 0) {
        const int64_t slot = a.slots[w.token];
        const bool in = slot >= 0 && slot < a.pages * a.page_size;
        int at;
        page = split_item(in ? slot : 0, a.page_size, at);
        row = at;
        if (!in) {
            if (slot >= 0 && reports && w.n > 0) atomicOr(a.err, kDevErrSlot);
            w.stored = 0;
        }
        if (s.scales) w.scales = s.scales + page * s.scale_page + row * s.scale_row + w.from * s.scale_head;
    }
    const int bytes = s.scales ? 1 : Elem<DT>::kBytes;
    w.out = static_cast<char*>(s.y) + (page * s.y_page + row * s.y_token + w.from * s.y_head) * bytes;
    w.step = s.y_head * bytes;
}

// The largest of a group's values, a NaN before any number.
template <int L> __device__ __forceinline__ float group_amax(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(u));
    }
    return v;
}

// An octet, as packed pairs in order, as codes: each times f0 and f1.
__device__ __forceinline__ uint2 octet_codes(const uint64_t (&z)[4], float f0, float f1) {
    uint64_t t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = f0 != 1.f ? f2_mul(z[i], f2_pack(f0, f0)) : z[i];
    return make_uint2(e4m3_pair(t[0], f1) | e4m3_pair(t[1], f1) << 16, e4m3_pair(t[2], f1) | e4m3_pair(t[3], f1) << 16);
}

// Two octets of a head row, z before its r, to a code row; one lane stores the scale.
__device__ __forceinline__ void store_codes(char* row, float* scale, int oa, int ob, const uint64_t (&za)[4],
                                            const uint64_t (&zb)[4], float amax, float r, bool first) {
    float f0, f1;
    const float s = quant_scale(amax, r, 0, f0, f1);
    if (oa >= 0) *reinterpret_cast<uint2*>(row + 8 * oa) = octet_codes(za, f0, f1);
    if (ob >= 0) *reinterpret_cast<uint2*>(row + 8 * ob) = octet_codes(zb, f0, f1);
    if (first) *scale = s;
}

template <int DT>
__device__ __forceinline__ void store_words(char* row, int oa, int ob, const uint32_t (&w)[2][Oct<DT>::kWords]) {
    constexpr int EB = Elem<DT>::kBytes, B = Oct<DT>::kBytes;
    octet_store<EB, Oct<DT>::kWords, true>(row + oa * B, w[0], oa >= 0 ? B : 0, false, false);
    octet_store<EB, Oct<DT>::kWords, true>(row + ob * B, w[1], ob >= 0 ? B : 0, false, false);
}

// Rows of whole octets, as rope_fwd_octets.
template <int DT, bool INTER, int L, bool CODES>
__global__ void __maxnreg__(96) append_octets(const __grid_constant__ AppendArgs a) {
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    constexpr int BATCH = rope_fwd_batch(DT);
    __shared__ Turns turns;
    const int li = threadIdx.x % L;
    griddep_wait();
    Work w = work_of(a, L);
    const AppendSet& set = w.set;
    int oa, ob;
    lane_octets<INTER>(li, a.D, a.R, oa, ob);
    const int rotated = rotated_pairs(a, li);
    const char* xb = static_cast<const char*>(set.x) + (w.token * set.x_token + w.from * set.x_head) * EB;
    const int64_t x_step = set.x_head * EB;
    uint32_t xw[BATCH][2][W];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) load16<DT>(xb + j * x_step, oa, ob, j < w.n, xw[j]);
    if (!w.rotate()) {  // values
        place<DT>(a, w, li == 0);
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            if (j >= a.chunk) break;
            if (CODES && set.scales) {
                uint64_t za[4], zb[4];
                octet_pairs<DT>(xw[j][0], za);
                octet_pairs<DT>(xw[j][1], zb);
                const float amax = group_amax<L>(max_magnitude(octet_amax<true>(za, 0, 8), octet_amax<true>(zb, 0, 8)));
                float* scale = w.scales + j * set.scale_head;
                if (j < w.stored) store_codes(w.out + j * w.step, scale, oa, ob, za, zb, amax, 1.f, li == 0);
            } else if (j < w.stored) {
                store_words<DT>(w.out + j * w.step, oa, ob, xw[j]);
            }
        }
        griddep_launch_dependents();
        return;
    }
    uint64_t pc[4], ps[4], qc[4], qs[4];
    load_gains<DT, INTER>(set, a.one, oa, ob, pc, qc);
    const int64_t pos = a.pos[w.token];
    place<DT>(a, w, li == 0);
    turns.fill(a, L);
    __syncthreads();
    {
        uint64_t c[4], s[4];
        turns.of_lane(a, li, pos, c, s);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            ps[k] = f2_mul(pc[k], s[k]);
            pc[k] = f2_mul(pc[k], c[k]);
            qs[k] = f2_neg(f2_mul(qc[k], s[k]));
            qc[k] = f2_mul(qc[k], c[k]);
        }
    }
    // rows with an infinity or a NaN are turned again (rope_fwd_octets)
    uint64_t sines = f2_add(ps[0], qs[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) sines = f2_add(sines, f2_add(ps[k], qs[k]));
    const float all = f2_sum(sines);
    const float finite = all == all ? __int_as_float(0x7f800000) : 0.f;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    // chunk is the same everywhere: the whole warp goes round as often (the sums see it)
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
        if (j >= a.chunk) break;
        uint64_t p[4], q[4];
        to_pairs<DT, INTER>(xw[j], p, q);
        uint64_t ss = f2_mul(p[0], p[0]);
#pragma unroll
        for (int k = 1; k < 4; ++k) ss = f2_fma(p[k], p[k], ss);
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = f2_fma(q[k], q[k], ss);
        const float sum = row_sum<L>(f2_sum(ss), nullptr);
        const float r = set.gamma ? row_rsqrt(sum, inv_d, a.eps) : 1.f;
        turn_pairs(p, q, pc, qs, qc, ps);
        if (rotated < 8 && j < w.n && !(sum < finite))
            turn_again<DT, INTER>(xb + j * x_step, oa, ob, rotated, p, q, pc, qs, qc, ps);
        char* row = w.out + j * w.step;
        if (CODES && set.scales) {
            // the octets' entries in order again
            uint64_t za[4], zb[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (INTER) {
                    float p0, p1, q0, q1;
                    f2_unpack(p[k], p0, p1);
                    f2_unpack(q[k], q0, q1);
                    (k < 2 ? za : zb)[2 * (k & 1)] = f2_pack(p0, q0);
                    (k < 2 ? za : zb)[2 * (k & 1) + 1] = f2_pack(p1, q1);
                } else {
                    za[k] = p[k];
                    zb[k] = q[k];
                }
            }
            const float amax = group_amax<L>(max_magnitude(octet_amax<true>(za, 0, 8), octet_amax<true>(zb, 0, 8)));
            if (j < w.stored) store_codes(row, w.scales + j * set.scale_head, oa, ob, za, zb, amax, r, li == 0);
        } else {
            const uint64_t r2 = f2_pack(r, r);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                p[k] = f2_mul(p[k], r2);
                q[k] = f2_mul(q[k], r2);
            }
            if (j < w.stored) store_pairs<DT, INTER>(row, oa, ob, p, q);
        }
    }
    griddep_launch_dependents();
}

// Halves whose octets do not meet octets: partners through shared memory, as rope_fwd_swap.
template <int DT, int L, bool CODES>
__global__ void __maxnreg__(128) append_swap(const __grid_constant__ AppendArgs a) {
    constexpr int W = Oct<DT>::kWords;
    constexpr int EB = Elem<DT>::kBytes;
    constexpr int BATCH = rope_fwd_batch(DT);
    __shared__ Turns turns;
    __shared__ float swaps[kFusedGroupThreads / 32 * 2 * kSwapFloats];
    const int li = threadIdx.x % L;
    griddep_wait();
    Work w = work_of(a, L);
    const AppendSet& set = w.set;
    const int oa = li < a.D / 8 ? li : -1, ob = li + L < a.D / 8 ? li + L : -1;
    const char* xb = static_cast<const char*>(set.x) + (w.token * set.x_token + w.from * set.x_head) * EB;
    const int64_t x_step = set.x_head * EB;
    uint32_t xw[BATCH][2][W];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
        load16<DT>(xb, oa, ob, j < w.n, xw[j]);
        xb += x_step;
    }
    uint64_t c[8], s[8];
    const int64_t pos = a.pos[w.token];
    place<DT>(a, w, li == 0);
    const Swap<L> swap(swaps, a, li);
    turns.fill(a, L);
    __syncthreads();
    swap.turns(turns, a, li, pos, false, c, s);
    {
        uint64_t g[8], gp[8];
        entry_gains<DT>(set, a.one, oa, ob, g);
        swap.partners(1, g, gp);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            c[k] = f2_mul(c[k], g[k]);
            s[k] = f2_mul(s[k], gp[k]);
        }
    }
    const float inv_d = 1.0f / static_cast<float>(a.D);
    char* row = w.out;
    float* scale = w.scales;
    for (int h = 0; h < a.chunk; h += BATCH) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            if (h + j >= a.chunk) break;
            uint64_t x[8], p[8];
            uint32_t raw[2][W];
#pragma unroll
            for (int k = 0; k < W; ++k) {
                raw[0][k] = xw[j][0][k];
                raw[1][k] = xw[j][1][k];
            }
            to_entries<DT>(xw[j], x);
            load16<DT>(xb, oa, ob, h + j + BATCH < w.n, xw[j]);
            xb += x_step;
            swap.partners(j & 1, x, p);
            uint64_t ss = f2_mul(x[0], x[0]);
#pragma unroll
            for (int k = 1; k < 8; ++k) ss = f2_fma(x[k], x[k], ss);
            float r = row_rsqrt(row_sum<L>(f2_sum(ss), nullptr), inv_d, a.eps);
            if (!set.gamma) r = 1.f;
            if (w.rotate()) {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = f2_fma(x[k], c[k], f2_mul(p[k], s[k]));
            }
            const bool live = h + j < w.stored;
            const uint64_t(&xa)[4] = *reinterpret_cast<const uint64_t(*)[4]>(&x[0]);
            const uint64_t(&xo)[4] = *reinterpret_cast<const uint64_t(*)[4]>(&x[4]);
            if constexpr (CODES) {
                const float amax = group_amax<L>(max_magnitude(octet_amax<true>(xa, 0, 8), octet_amax<true>(xo, 0, 8)));
                if (set.scales && live) store_codes(row, scale, oa, ob, xa, xo, amax, r, li == 0);
            }
            if (!set.scales && live) {
                if (w.rotate()) {
                    const uint64_t r2 = f2_pack(r, r);
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = f2_mul(x[k], r2);
                    store_entries<DT>(row, oa, ob, x);
                } else {
                    store_words<DT>(row, oa, ob, raw);
                }
            }
            row += w.step;
            if (scale) scale += set.scale_head;
        }
    }
    griddep_launch_dependents();
}

// Any D, R and alignment, entry by entry, as rope_pairs.
template <int DT, int L, int PK, bool CODES>
__global__ void __launch_bounds__(kFusedGroupThreads) append_pairs(const __grid_constant__ AppendArgs a) {
    constexpr int EB = Elem<DT>::kBytes;
    const int li = threadIdx.x % L;
    griddep_wait();
    int ca[PK], cb[PK];
    lane_pairs<L, PK>(li, a, a.interleaved != 0, ca, cb);
    const float inv_d = 1.0f / static_cast<float>(a.D);
    Work w = work_of(a, L);
    const AppendSet& set = w.set;
    place<DT>(a, w, li == 0);
    const int64_t pos = a.pos[w.token];
    float c[PK], s[PK];
#pragma unroll
    for (int k = 0; k < PK; k += 2) {
        const int i0 = li + L * k, i1 = i0 + L, half = a.R / 2;
        c[k] = c[k + 1] = 1.f;
        s[k] = s[k + 1] = 0.f;
        if (i0 < half) {
            uint64_t c2, s2;
            turn_pair(phase_at(turns_per_position(a.inv_freq[i0]), pos),
                      i1 < half ? phase_at(turns_per_position(a.inv_freq[i1]), pos) : 0, a.mscale, a.mscale, c2, s2);
            f2_unpack(c2, c[k], c[k + 1]);
            f2_unpack(s2, s[k], s[k + 1]);
        }
    }
    const char* gb = static_cast<const char*>(set.gamma);
    float g[2 * PK];
#pragma unroll
    for (int j = 0; j < 2 * PK; ++j) {
        const int col = j & 1 ? cb[j / 2] : ca[j / 2];
        g[j] = gb && col >= 0 ? entry<DT>(gb, col) + a.one : 1.f;
    }
    const char* xr = static_cast<const char*>(set.x) + (w.token * set.x_token + w.from * set.x_head) * EB;
    const int64_t x_step = set.x_head * EB;
    float ahead[2 * PK];  // the next head's entries
    const auto load = [&](const char* row, bool live) {
#pragma unroll
        for (int j = 0; j < 2 * PK; ++j) {
            const int col = j & 1 ? cb[j / 2] : ca[j / 2];
            ahead[j] = live && col >= 0 ? entry<DT>(row, col) : 0.f;
        }
    };
    load(xr, w.n > 0);
    for (int h = 0; h < a.chunk; ++h, xr += x_step) {
        float x[2 * PK];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 2 * PK; ++j) {
            x[j] = ahead[j];
            ss = fmaf(x[j], x[j], ss);
        }
        load(xr + x_step, h + 1 < w.n);
        const float r = gb ? row_rsqrt(group_sum<L>(ss), inv_d, a.eps) : 1.f;
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < PK; ++k) {
            if (w.rotate()) {
                float z0 = x[2 * k], z1 = x[2 * k + 1];
                if (gb) {
                    // of codes the r is left out, as in the octets
                    const float f = set.scales ? 1.f : r;
                    z0 = (z0 * f) * g[2 * k];
                    z1 = (z1 * f) * g[2 * k + 1];
                }
                const bool rotated = li + L * k < a.R / 2;
                x[2 * k] = rotated ? z0 * c[k] - z1 * s[k] : z0;
                x[2 * k + 1] = rotated ? z1 * c[k] + z0 * s[k] : z1;
            }
            amax = max_magnitude(max_magnitude(amax, x[2 * k]), x[2 * k + 1]);
        }
        float f0 = 1.f, f1 = 1.f;
        if constexpr (CODES) {
            amax = group_amax<L>(amax);
            if (set.scales) {
                const float scale = quant_scale(amax, r, 0, f0, f1);
                if (h < w.stored && li == 0) w.scales[h * set.scale_head] = scale;
            }
        }
        char* row = w.out + h * w.step;
#pragma unroll
        for (int j = 0; j < 2 * PK; ++j) {
            const int col = j & 1 ? cb[j / 2] : ca[j / 2];
            if (h >= w.stored || col < 0) continue;
            if (CODES && set.scales) {
                row[col] = static_cast<char>(e4m3_pair(f2_pack(x[j] * f0, 0.f), f1));
            } else if (w.rotate()) {
                Elem<DT>::st(row, col, x[j]);
            } else if constexpr (EB == 2) {  // values as they are, the payloads of NaNs too
                reinterpret_cast<uint16_t*>(row)[col] = reinterpret_cast<const uint16_t*>(xr)[col];
            } else {
                reinterpret_cast<uint32_t*>(row)[col] = reinterpret_cast<const uint32_t*>(xr)[col];
            }
        }
    }
    griddep_launch_dependents();
}

template <int DT, bool CODES> const void* kernel_for(const RopePlan& p) {
#define RMSNORM_APPEND(L)                                                                                              \
    if (p.lanes == L) {                                                                                                \
        if (p.rows == kRopeNeighbours) return reinterpret_cast<const void*>(&append_octets<DT, true, L, CODES>);      \
        if (p.rows == kRopeHalves) return reinterpret_cast<const void*>(&append_octets<DT, false, L, CODES>);         \
        if (p.rows == kRopeSwap) return reinterpret_cast<const void*>(&append_swap<DT, L, CODES>);                    \
    }
    RMSNORM_APPEND(4)
    RMSNORM_APPEND(8)
    RMSNORM_APPEND(16)
    RMSNORM_APPEND(32)
#undef RMSNORM_APPEND
    switch (p.lanes) {
    case 8: return reinterpret_cast<const void*>(&append_pairs<DT, 8, 4, CODES>);
    case 16: return reinterpret_cast<const void*>(&append_pairs<DT, 16, 4, CODES>);
    default: break;
    }
    return p.pairs <= 4 ? reinterpret_cast<const void*>(&append_pairs<DT, 32, 4, CODES>)
                        : reinterpret_cast<const void*>(&append_pairs<DT, 32, 8, CODES>);
}

}  // namespace

const void* append_kernel(const RopePlan& p, bool codes) {
    switch (p.dtype) {
    case kF32: return codes ? kernel_for<kF32, true>(p) : kernel_for<kF32, false>(p);
    case kF16: return codes ? kernel_for<kF16, true>(p) : kernel_for<kF16, false>(p);
    case kBF16: return codes ? kernel_for<kBF16, true>(p) : kernel_for<kBF16, false>(p);
    default: return nullptr;
    }
}

}  // namespace rmsnorm
