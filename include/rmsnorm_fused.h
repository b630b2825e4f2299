/*
 * rmsnorm_fused.h -- C ABI of the operators that stand around an RMSNorm in a
 * transformer block, one kernel each (two with a gradient of the weight):
 *
 *   rmsnorm_add_fwd / _bwd    dropout, residual addition and RMSNorm, with gradients
 *   rmsnorm_quant_fwd         residual addition, RMSNorm and an 8-bit output with scales
 *   rmsnorm_rope_fwd / _bwd   RMSNorm of attention heads and rotary positions, with gradients
 *
 * Conventions are those of rmsnorm.h: device pointers on the current device, the
 * caller owns every buffer and the stream, no allocation, all checks on the host
 * before any launch, fp32 arithmetic whatever the I/O dtype, status codes. Rows
 * are ld* elements apart (ld* >= N; the gaps are neither read nor written). Any
 * element-aligned pointer and pitch works; the wide path wants every row to start
 * on a 16-byte boundary and N to be a multiple of 8, other rows are moved in
 * 16-byte words that are shifted together.
 *
 * In place: every row is read before it is written, so an output may be an input
 * of the same shape, dtype, pointer and pitch (h on residual, y on x, dresidual on
 * dy or dh, rotated heads on the heads). No other overlap is allowed; two outputs at
 * one address whose values differ are refused, and so are an output's rows that overlap
 * and an output that starts where an input of another pitch, the weight (of several rows) or
 * another set's heads do.
 */
#ifndef RMSNORM_FUSED_H
#define RMSNORM_FUSED_H

#include "rmsnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Forward of the residual branch. For each row
 *
 *     h = D(x) + residual             rounded to dtype: the residual stream
 *     r = 1 / sqrt(mean(h^2) + eps)
 *     y = h * r * g                   g = gamma, or 1 + gamma with offset
 *
 * The norm is that of the rounded h. D is dropout: with t = round(65536 * p), D(x)
 * = x * 65536 / (65536 - t) where an element is kept and 0 where it is dropped,
 * which is where its 16-bit number is below t. The numbers are a function of the
 * seed, the offset and the element's row and column: the low and high halves, in
 * order, of the words of Philox4x32-10 with counter {column / 8, row, offset low,
 * offset high} and key {seed low, seed high}, one call for eight columns. No mask
 * is stored; the backward draws the same numbers.
 *
 * residual may be NULL (h = D(x)), h may be NULL (not written), rstd may be NULL
 * (float32[M], kept for the backward). dropout_p is in [0, 1]; 0 (or less than
 * 2^-17) is no dropout. rng: {seed, offset}, two 64-bit integers in DEVICE memory,
 * read when the kernel runs, so that a captured graph draws new numbers after they
 * are changed; required with dropout, ignored without. rng_used: NULL, or room for
 * the two values that this call used (written only with dropout), for a backward
 * that runs after rng has moved on. Calls that draw from the same seed want
 * different offsets.
 */
rmsnorm_status rmsnorm_add_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldres, const void* gamma,
                               void* h, int64_t ldh, void* y, int64_t ldy, float* rstd, int64_t M, int64_t N,
                               float eps, rmsnorm_dtype dtype, int offset, float dropout_p,
                               const uint64_t* rng, uint64_t* rng_used, rmsnorm_stream_t stream);

/*
 * Backward of rmsnorm_add_fwd: for the cotangents dy of y and dh of h (dh may be
 * NULL: zero), with n = h * rstd and u = dy * g,
 *
 *     dresidual = dh + rstd * (u - n * mean(u * n))
 *     dx        = dresidual * 65536 / (65536 - t) where kept, 0 where dropped
 *                 (before dresidual is rounded)
 *     dgamma    = sum over rows of dy * n
 *
 * h and rstd are the forward's. dx and dresidual may each be NULL; without dropout
 * they are equal. dgamma is deterministic, as that of rmsnorm_bwd: fp32 partial
 * sums over fixed rows in `workspace` (at least rmsnorm_add_bwd_workspace_size
 * bytes, 16-byte aligned, scratch, not shared by calls that overlap on the GPU),
 * then a column reduction in a fixed order. M == 0 writes dgamma = 0.
 */
size_t rmsnorm_add_bwd_workspace_size(int64_t M, int64_t N, rmsnorm_dtype dtype);
rmsnorm_status rmsnorm_add_bwd(const void* dy, int64_t lddy, const void* dh, int64_t lddh, const void* h, int64_t ldh,
                               const void* gamma, const float* rstd, void* dx, int64_t lddx, void* dresidual,
                               int64_t lddres, void* dgamma, int64_t M, int64_t N, rmsnorm_dtype dtype, int offset,
                               float dropout_p, const uint64_t* rng, void* workspace, size_t workspace_bytes,
                               rmsnorm_stream_t stream);

/*
 * Forward for 8-bit matrix products: h and y as in rmsnorm_add_fwd without dropout,
 * y kept in fp32 and written as e4m3 codes (1 sign, 4 exponent, 3 fraction bits,
 * largest 448) with a float32 scale per row (group 0) or per group of 32, 64 or
 * 128 columns (the row's last group may be short):
 *
 *     scale = max(amax(|y|) / 448, 2^-126)      pow2: rounded up to a power of two
 *     code  = y / scale, rounded to nearest-even
 *
 * (fp32's y / scale: one that lies half way between two codes may become either of them.)
 * codes: uint8[M rows, pitch ldcodes]; scales: float32[M rows, pitch ldscales],
 * one per row or ceil(N / group). residual and h may be NULL, each on its own. A
 * group with a NaN gets a NaN scale; one with an infinity an infinite scale and
 * codes of 0 and NaN. h * g is formed before r is known: where that passes fp32's
 * range (2^128), y counts as infinite.
 */
rmsnorm_status rmsnorm_quant_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldres, const void* gamma,
                                 void* h, int64_t ldh, void* codes, int64_t ldcodes, float* scales, int64_t ldscales,
                                 int64_t M, int64_t N, float eps, rmsnorm_dtype dtype, int offset, int group, int pow2,
                                 rmsnorm_stream_t stream);

#define RMSNORM_ROPE_MAX_D 512
#define RMSNORM_ROPE_MAX_SETS 2
#define RMSNORM_ROPE_MAX_HEADS 65536

/*
 * Heads of one kind (a model's query heads, its key heads): entry d of head j of
 * token t is at x[t * x_token + j * x_head + d], strides in elements, each at least
 * D where there is more than one token or head; of an output (y, dx) also all heads of
 * a token within a token's stride, or all tokens of a head within a head's. gamma[D], shared by the heads, or
 * NULL for the rotation without a norm. y: the output, with its own strides.
 */
typedef struct {
    const void* x;
    int64_t x_token, x_head;
    const void* gamma;
    void* y;
    int64_t y_token, y_head;
    int64_t heads;
} rmsnorm_rope_heads;

/* The same for the backward: dy of y, the forward's x, dx, and dgamma[D] (ignored
 * where gamma is NULL, as x is there). */
typedef struct {
    const void* dy;
    int64_t dy_token, dy_head;
    const void* x;
    int64_t x_token, x_head;
    const void* gamma;
    void* dx;
    int64_t dx_token, dx_head;
    void* dgamma;
    int64_t heads;
} rmsnorm_rope_heads_bwd;

/*
 * RMSNorm of every head row (z = x * r * g, r over its D entries; z = x where gamma
 * is NULL), and the rotation of its first rotary_dim entries: for each pair (a, b)
 *
 *     y_a = z_a * cos - z_b * sin,  y_b = z_b * cos + z_a * sin
 *
 * with cos and sin of positions[t] * inv_freq[i], both times mscale. Pair i is the
 * entries (2i, 2i + 1) with interleaved = 1, (i, i + rotary_dim / 2) with 0. The
 * entries from rotary_dim on are z. One to RMSNORM_ROPE_MAX_SETS sets, rotated
 * alike, in one launch. positions: int64[T], any values; inv_freq:
 * float64[rotary_dim / 2], finite, in radians per position: a scaled context is a
 * matter of the frequencies (and mscale) given. Angles are reduced in 64-bit fixed
 * point: with frequencies below 4 by that an angle is off by less than 2^-31 of a turn at
 * any position up to 2^32 (and by position * 2^-63 of a turn at others). What is left of a
 * quarter turn is rounded to fp32, and its sine and cosine come out within 2^-21 of
 * themselves. x * g is formed before r, as above. 1 <= D <= RMSNORM_ROPE_MAX_D,
 * rotary_dim even, 2 <= rotary_dim <= D; T may be 0; at most
 * RMSNORM_ROPE_MAX_HEADS heads in all sets.
 */
rmsnorm_status rmsnorm_rope_fwd(const rmsnorm_rope_heads* sets, int nsets, const int64_t* positions, int64_t T,
                                int64_t D, int64_t rotary_dim, const double* inv_freq, int interleaved, float mscale,
                                float eps, rmsnorm_dtype dtype, int offset, rmsnorm_stream_t stream);

/*
 * Backward: v = dy rotated back, u = v * g, n = x * r (r computed again from x),
 * dx = r * (u - n * mean(u * n)), dgamma = sum over tokens and heads of v * n,
 * deterministic through `workspace` as in rmsnorm_add_bwd (it may be NULL when no
 * set has a gamma). heads: of all sets. T == 0 writes dgamma = 0.
 */
size_t rmsnorm_rope_bwd_workspace_size(int64_t T, int64_t heads, int64_t D, rmsnorm_dtype dtype);
rmsnorm_status rmsnorm_rope_bwd(const rmsnorm_rope_heads_bwd* sets, int nsets, const int64_t* positions, int64_t T,
                                int64_t D, int64_t rotary_dim, const double* inv_freq, int interleaved, float mscale,
                                float eps, rmsnorm_dtype dtype, int offset, void* workspace, size_t workspace_bytes,
                                rmsnorm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RMSNORM_FUSED_H */
