/*
 * rmsnorm_serving.h -- C ABI of the operators between an RMSNorm and an attention in
 * serving:
 *
 *   rmsnorm_quant_weight   a weight as e4m3 codes with a scale per block of 128 x 128
 *   rmsnorm_quant_matmul   the product of rmsnorm_quant_fwd's codes with such a weight
 *   rmsnorm_rope_append    head norm and rotation of queries and keys, with keys and values
 *                          written to the rows of a paged cache
 *
 * Conventions are those of rmsnorm.h: device pointers on the current device, the caller owns
 * every buffer and the stream, no allocation, no workspace, all checks on the host before any
 * launch, status codes. None of them has a gradient. Rows are ld* elements apart (ld* >= the
 * row; the gaps are not written and what they hold does not matter), and any element-aligned
 * pointer and pitch works; the fast paths want rows on 16-byte boundaries. Other rows are read in
 * whole 16-byte words, each with a byte of the row at least.
 */
#ifndef RMSNORM_SERVING_H
#define RMSNORM_SERVING_H

#include "rmsnorm_fused.h"

#ifdef __cplusplus
extern "C" {
#endif

#define RMSNORM_MATMUL_MAX 1048576 /* most rows and columns of a weight */
#define RMSNORM_MATMUL_BLOCK 128

/*
 * The weight w[N, K] (dtype) as e4m3 codes (uint8[N rows, pitch ldcodes]; 1 sign, 4 exponent, 3
 * fraction bits, largest 448) with a float32 scale per block of 128 x 128, the last ones
 * of a row and column short (scales[ceil(N / 128) rows, pitch ldscales >= ceil(K / 128)]):
 *
 *     scale = max(amax(|w|) / 448, 2^-126)      pow2: rounded up to a power of two
 *     code  = w / scale, rounded to nearest-even
 *
 * with both quotients rounded exactly. A block with a NaN gets a NaN scale, one with an
 * infinity an infinite scale and codes of 0 and NaN. N may be 0. The outputs must not overlap
 * the weight or each other.
 */
rmsnorm_status rmsnorm_quant_weight(const void* w, int64_t ldw, void* codes, int64_t ldcodes, float* scales,
                                    int64_t ldscales, int64_t N, int64_t K, rmsnorm_dtype dtype, int pow2,
                                    rmsnorm_stream_t stream);

/*
 * The product of 8-bit rows with an 8-bit weight:
 *
 *     y[m, n] = sum over k of (a[m, k] a_scales[m, k / group]) (b[n, k] b_scales[n / 128, k / 128]) + bias[n]
 *
 * a: e4m3 codes of M rows of K with scales per 128 columns (group 128: a_scales[M rows, pitch
 * ldas >= ceil(K / 128)]) or per row (group 0: ldas >= 1), as rmsnorm_quant_fwd writes them; b:
 * [N, K] with scales per block, as rmsnorm_quant_weight writes them. y[M, N] is fp32, fp16
 * or bf16 (dtype), and bias[N], which may be NULL, of the same type. The products within a block
 * of 128 columns are summed by the tensor cores in fp32, the blocks, times the product of
 * their two scales, in fp32; one rounding to y's type. A pair of scales whose product passes
 * fp32's range counts as infinite, or as 0 below it. A result depends on the operands, their
 * alignment, M, N, K and the device (which choose the order of the sums), not on the run.
 * 1 <= N, K <= RMSNORM_MATMUL_MAX; M may be 0. y must not overlap an operand.
 */
rmsnorm_status rmsnorm_quant_matmul(const void* a, int64_t lda, const float* a_scales, int64_t ldas, const void* b,
                                    int64_t ldb, const float* b_scales, int64_t ldbs, const void* bias, void* y,
                                    int64_t ldy, int64_t M, int64_t N, int64_t K, rmsnorm_dtype dtype, int group,
                                    rmsnorm_stream_t stream);

/*
 * Heads of one kind for a paged cache, a model's keys or its values: entry d of head j of
 * token t is at x[t * x_token + j * x_head + d] (strides in elements, as in
 * rmsnorm_rope_heads), gamma[D] the weight of the keys' norm or NULL (always NULL of
 * values). Entry d of head j of row i of page p of the cache is at rows[p * page + i * row + j *
 * head + d], in any order of the three strides that keeps the rows apart. scales NULL: rows
 * are of the call's dtype. Else they are e4m3 codes (uint8), with the head row's float32 scale
 * at scales[p * scale_page + i * scale_row + j * scale_head]: scale = max(max|z| / 448, 2^-126),
 * code = z / scale as in rmsnorm_quant_fwd, non-finite entries too.
 */
typedef struct {
    const void* x;
    int64_t x_token, x_head;
    const void* gamma;
    void* rows;
    int64_t page, row, head;
    float* scales;
    int64_t scale_page, scale_row, scale_head;
    int64_t heads;
} rmsnorm_cache_heads;

/*
 * One step of serving before an attention: queries and keys are normalised and rotated as by
 * rmsnorm_rope_fwd (same arguments), queries go to q's y, and keys and values (as they are) go
 * to slot slots[t] of their caches: row slots[t] % page_size of page slots[t] / page_size,
 * of `pages` pages. A negative slot (a padded token) stores nothing; its query is
 * rotated all the same. A slot behind the last stores nothing and sets bit 2 of the device
 * error word (rmsnorm_device_error). Slots of one call that are not negative must be
 * distinct: of rows that share one, what remains is unspecified. Rows that no slot names
 * are not touched. The queries' output may be the queries (pointer and strides) or lie between
 * the rows of other heads; one that meets them otherwise is refused. slots: int64[T]. q may be NULL
 * (a prompt's keys alone), and v may be (keys that serve as values). The caches may be interleaved parts of one tensor of
 * the same strides; they must not overlap the heads, the weights or each other otherwise. Values
 * are copied bit by bit where their cache has no scales.
 */
rmsnorm_status rmsnorm_rope_append(const rmsnorm_rope_heads* q, const rmsnorm_cache_heads* k,
                                   const rmsnorm_cache_heads* v, const int64_t* slots, int64_t pages,
                                   int64_t page_size, const int64_t* positions, int64_t T, int64_t D,
                                   int64_t rotary_dim, const double* inv_freq, int interleaved, float mscale, float eps,
                                   rmsnorm_dtype dtype, int offset, rmsnorm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RMSNORM_SERVING_H */
