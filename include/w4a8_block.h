/*
 * w4a8_block.h -- C ABI of the operators that stand between the W4A8 linears of a decoder
 * layer on AMD MI355X (gfx950): the RMS norm that feeds them, its backward, rotary
 * positions, an 8-bit paged cache of keys and values, and attention over it.  They are
 * part of libw4a8.so; the linears themselves are in w4a8.h, whose status codes these
 * entries return.
 *
 * Conventions (those of w4a8.h):
 *   - All buffers are DEVICE pointers owned by the caller.  The library allocates, frees
 *     and retains nothing, keeps no state between calls and never synchronises the
 *     stream.  Structs passed by pointer are HOST memory, read during the call only.
 *   - `stream` is a hipStream_t (NULL = the null stream).  Work is enqueued on it in
 *     order; calls on different streams are independent.
 *   - Arguments are validated on the host before anything is launched; a call that
 *     returns an error has enqueued nothing and written nothing.  Lengths, page numbers
 *     and row offsets that lie in device memory cannot be seen by the host: the kernels
 *     bound them themselves (stated at each entry), so none of them can reach memory
 *     outside the buffers described by the arguments.
 *   - A call that would take 2^24 blocks or more is refused with W4A8_ERR_SHAPE.
 *   - Return value: W4A8_OK (0) or one of the W4A8_ERR_* codes of w4a8.h.
 *   - Dense tensors are row-major.  Activation tensors [T, heads, head_dim] have dense
 *     heads and a token stride in elements, so the queries, keys and values of one
 *     projection's output [T, (Hq + 2 Hkv) * head_dim] are passed as they lie.
 *   - Alignment: 16 bytes for activations, streams, weights, codes and workspaces; 4 for
 *     scales, rstd, positions, lengths and tables.
 */
#ifndef W4A8_BLOCK_H
#define W4A8_BLOCK_H

#include <stdint.h>

#include "w4a8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of the residual stream. */
enum w4a8_stream_type { W4A8_STREAM_BF16 = 0, W4A8_STREAM_F32 = 1 };

#define W4A8_NORM_MAX_K 16384     /* columns of a normalised row */
#define W4A8_ROPE_MAX_AXES 4
#define W4A8_ROPE_MAX_HEAD_DIM 256

/*
 * rmsnorm_quant_act -- residual addition, RMS norm, and the activation step of the next
 * W4A8 linear (rotate_quant_act) in one pass, for M rows of K columns:
 *   h[m, k] = residual[m, k] + x[m, k]   in fp32, rounded once to the stream's type
 *   rstd[m] = 1 / sqrt(mean_k(h^2) + eps)
 *   y[m, k] = h * rstd * weight[k]       in fp32 (not rounded before the rotation)
 *   v       = y rotated as in rotate_quant_act (every 256 columns times H4^(x4) / 16)
 *   xs[m]   = max_k |v| / qmax (1.0 for a zero row), xq = rint(v / xs) in -qmax..qmax
 * The norm is that of the stored (rounded) h, so the backward needs nothing else.  Sums
 * and the rotation are in fp32.  A row whose sum of squares is not finite (an inf or NaN
 * input, or an overflow of fp32) gets rstd = NaN, xs = NaN, codes 0 and y = NaN.
 *
 *   x            in   bf16 bits [M, K]
 *   residual     in   [M, K] of stream_type, or NULL: h is x itself and h must be NULL
 *   weight       in   float [K]
 *   M, K              0 <= M < 2^22; 256 <= K <= W4A8_NORM_MAX_K, K % 256 == 0
 *   eps               > 0, finite
 *   rot_block         must be 256;  qmax 1..127
 *   h            out  NULL, or [M, K] of stream_type; may be `residual` itself
 *   rstd         out  NULL, or float [M] (kept for rmsnorm_grad)
 *   y            out  NULL, or bf16 bits [M, K]: y rounded to nearest even (a final norm)
 *   xq, xs       out  int8 [M, K] and float [M], or both NULL when y is wanted alone
 * h apart, outputs may not overlap inputs.
 */
int rmsnorm_quant_act(const void* x, const void* residual, int32_t stream_type, const float* weight, int64_t M,
                      int64_t K, float eps, int32_t rot_block, int32_t qmax, void* h, float* rstd, void* y,
                      int8_t* xq, float* xs, void* stream);

/*
 * rmsnorm_grad -- the backward of rmsnorm_quant_act, straight through the quantiser:
 *   gy[m, k] = grad rotated back (the rotation is its own inverse), or grad if rot_block is 0
 *   u        = gy * weight,  c[m] = rstd^2 * mean_k(u * h)
 *   dx       = grad_h + rstd * (u - h * c)       the gradient of x and of residual alike
 *   dweight  = sum_m gy * h * rstd               overwritten, summed in a fixed order
 * all in fp32, dx rounded once to the stream's type.
 *
 *   grad         in   bf16 bits [M, K]: with rot_block 256 the gradient of the rotated
 *                     activation (what w4a8_grad_input gives), with rot_block 0 that of y
 *   h            in   [M, K] of stream_type (x, with W4A8_STREAM_BF16, if there was no residual)
 *   rstd         in   float [M]
 *   grad_h       in   NULL, or [M, K] of stream_type: the gradient that reached h otherwise
 *   dx           out  [M, K] of stream_type; may be grad_h itself
 *   dweight      out  NULL, or float [K]
 *   workspace         with dweight: rmsnorm_grad_workspace(M, K) bytes at least, else NULL, 0
 */
int rmsnorm_grad(const void* grad, const void* h, int32_t stream_type, const float* rstd, const float* weight,
                 const void* grad_h, int64_t M, int64_t K, int32_t rot_block, void* dx, float* dweight,
                 void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that rmsnorm_grad needs for dweight; 0 for sizes it refuses. */
int64_t rmsnorm_grad_workspace(int64_t M, int64_t K);

/*
 * Rotary positions with one to four axes (time, height, width, ...).  A head's first
 * rotary_dim elements are rotary_dim / 2 pairs; pair p belongs to one axis (the first
 * sections[0] pairs to axis 0, the next sections[1] to axis 1, ...) and is turned by the
 * angle pos[axis, t] * inv_freq[p] (the exact product, reduced in fp64):
 *   (a, b) -> (a cos - b sin, b cos + a sin).
 * Elements past rotary_dim are passed through.
 */
typedef struct w4a8_rope {
    const int32_t* pos;                      /* device [axes, T], rows pos_stride apart */
    int64_t pos_stride;                      /* >= T */
    const float* inv_freq;                   /* device float [rotary_dim / 2] */
    int32_t rotary_dim;                      /* multiple of 16, 16..head_dim */
    int32_t axes;                            /* 1..W4A8_ROPE_MAX_AXES */
    int32_t sections[W4A8_ROPE_MAX_AXES];    /* pairs of each axis, >= 0; sum rotary_dim / 2 */
    int32_t interleaved;                     /* 0: pair p is (p, p + rotary_dim / 2); 1: (2p, 2p + 1) */
} w4a8_rope;

/*
 * rope_axes -- rotates every head of x.  inverse != 0 turns by the negative angles: the
 * rotation's transpose, hence its inverse and its backward.
 *   x          in   bf16 bits, T tokens of `heads` dense heads, x_stride elements apart
 *   head_dim        multiple of 16, 16..W4A8_ROPE_MAX_HEAD_DIM; T >= 0, heads >= 1
 *   x_stride        >= heads * head_dim, multiple of 8 (so is out_stride)
 *   out        out  bf16 bits, fp32 arithmetic rounded once; may be x itself (same stride)
 */
int rope_axes(const void* x, int64_t T, int32_t heads, int32_t head_dim, int64_t x_stride, const w4a8_rope* rope,
              int32_t inverse, void* out, int64_t out_stride, void* stream);

/*
 * The 8-bit paged cache.  A page holds page_tokens consecutive tokens of one sequence for
 * all heads; keys and values are int8 codes with one fp32 scale for each page and head:
 *   key[t, d]   = k[page, head, t % page_tokens, d] * k_scale[page, head]
 *   value[t, d] = v[page, head, d, t % page_tokens] * v_scale[page, head]
 * (values lie transposed: the contraction over tokens then reads 16 codes at a time).
 * table[b, i] is the page of tokens i * page_tokens .. of sequence b.  A scale of 0 stands
 * for a page of zeros, a NaN scale for a page that was given an inf or NaN.
 */
typedef struct w4a8_kv8 {
    int8_t* k;                 /* device [pages, heads, page_tokens, head_dim] */
    int8_t* v;                 /* device [pages, heads, head_dim, page_tokens] */
    float* k_scale;            /* device [pages, heads], >= 0 */
    float* v_scale;            /* device [pages, heads], >= 0 */
    int64_t pages;             /* >= 1 */
    int32_t heads;             /* >= 1, key and value heads */
    int32_t head_dim;          /* 64 or 128 */
    int32_t page_tokens;       /* 16, 32, 64 or 128 */
    int32_t table_stride;      /* >= 1, pages of a table row */
    const int32_t* table;      /* device [B, table_stride]; may be NULL if B is 0 */
} w4a8_kv8;

/*
 * kv8_append -- puts new tokens of B sequences at the end of their cached ones, and
 * rotates their keys, and optionally their queries, on the way (one launch).
 * Rows q_start[b] .. q_start[b + 1] - 1 of k, v (and q) are the new tokens of sequence b,
 * which held ctx_len[b] tokens before.  For every page they touch, head, and each of keys
 * (after rotation, in fp32) and values:
 *   scale' = max(scale if the page holds earlier tokens else 0, max |new| / 127)
 *   a new token's codes:      rint(x / scale') (0 if scale' is 0)
 *   earlier tokens' codes:    rint(code * (scale / scale')) if scale' > scale, else kept
 *   positions past the last:  0 in a page that holds no earlier tokens, else left
 * An inf or NaN among the new values makes scale' NaN and the codes 0; NaN stays.
 *
 *   cache             the cache; its codes and scales are updated in place
 *   ctx_len      in   int32 [B], tokens held before the call
 *   q_start      in   int32 [B + 1], ascending
 *   B, T              sequences >= 0, rows of k, v, q >= 0
 *   max_new           upper bound of the new tokens of a sequence; tokens past it are not
 *                     appended
 *   k, v         in   bf16 bits, T tokens of cache->heads heads, k_stride / v_stride apart
 *   q            in   NULL, or bf16 bits, T tokens of q_heads heads, q_stride apart
 *   rope              NULL (keys stored and queries copied as they are) or the rotation
 *   q_out        out  bf16 bits [T, q_heads, head_dim], out_stride apart; may be q itself
 * Rows outside 0..T, positions outside a table row and page numbers outside 0..pages - 1
 * are skipped.  Two sequences must not share a page that the call appends to.
 */
int kv8_append(const w4a8_kv8* cache, const int32_t* ctx_len, const int32_t* q_start, int64_t B, int64_t T,
               int64_t max_new, const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q,
               int32_t q_heads, int64_t q_stride, const w4a8_rope* rope, void* q_out, int64_t out_stride,
               void* stream);

/*
 * kv8_attention -- softmax attention of the last tokens of B sequences over their cached
 * ones.  Query row i of sequence b (row q_start[b] + i of q, n = q_start[b + 1] -
 * q_start[b] of them) stands at position p = kv_len[b] - n + i.  It sees the keys
 * j < kv_len[b] with j <= p if causal, and j > p - window if window > 0 (also then j <= p
 * only if causal).  Query head h reads cache head h / (q_heads / heads):
 *   out = sum_j w_j value_j / sum_j w_j,  w_j = exp(scale * q . key_j - max),
 *   lse = log sum_j exp(scale * q . key_j)
 * A row that sees no key gets out 0 and lse -inf.  Codes are exact in bf16, and so are the
 * queries: scores are exact products summed in fp32; the weights, relative to the largest
 * seen so far (as is the value scale), are rounded to fp16 (11 bits; below 2^-29 of the
 * largest in steps of 2^-39) for the product with the values, which sums in fp32.  The
 * sum of the weights, in fp32, has no part in that scale: it is of the weights as rounded (the
 * rounding then nearly cancels), or unrounded where a small value scale leaves fp16 too few bits.
 * out is rounded once to bf16.  A masked key or value never reaches the result, whatever it
 * holds; a page of NaN scales that a row sees makes the row NaN.
 *
 *   q            in   bf16 bits, T tokens of q_heads heads, q_stride elements apart
 *   q_heads           multiple of cache->heads
 *   kv_len       in   int32 [B], cached tokens (the new ones among them); bounded by the
 *                     table row's capacity
 *   q_start      in   int32 [B + 1], ascending, bounded by T
 *   max_new           upper bound of n; further rows of a sequence are not computed (rows of q that
 *                     are not computed leave out and lse as they are)
 *   max_kv            upper bound of kv_len, used for the division of work only.  It and max_new
 *                     divide the whole call: single tokens over long contexts beside a
 *                     prompt run undivided, and are much faster in a call of their own
 *   scale             > 0, finite
 *   out          out  bf16 bits [T, q_heads, head_dim], out_stride apart
 *   lse          out  NULL, or float [T, q_heads]
 *   workspace         kv8_attention_workspace(...) bytes at least (NULL if that is 0)
 * A page number outside 0..pages - 1 hides its tokens.
 * Refused with W4A8_ERR_SHAPE: 2^24 query rows or more, min(T, B * max_new) * q_heads, or as many
 * row tiles, B * heads * ceil(max_new * (q_heads / heads) / r), with r = 16 for less than 64
 * rows of a sequence and cache head and 128 for more.
 */
int kv8_attention(const void* q, int32_t q_heads, int64_t q_stride, const w4a8_kv8* cache, const int32_t* kv_len,
                  const int32_t* q_start, int64_t B, int64_t T, int64_t max_new, int64_t max_kv, float scale,
                  int32_t causal, int64_t window, void* out, int64_t out_stride, float* lse, void* workspace,
                  int64_t workspace_bytes, void* stream);

/* Bytes of workspace that kv8_attention needs (0 where it divides no context). */
int64_t kv8_attention_workspace(int64_t B, int64_t T, int64_t max_new, int64_t max_kv, int32_t q_heads,
                                int32_t kv_heads, int32_t head_dim);

/* Version of this header's entries (incremented on any signature change). */
int w4a8_block_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* W4A8_BLOCK_H */
