// C ABI entry points of include/w4a8_block.h: host validation without any HIP call, then
// the launch on the caller's stream.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/w4a8_block.h"
#include "kv8_plan.hpp"

namespace w4a8 {
hipError_t launch_rmsnorm_quant(const void* x, const void* residual, int stream_f32, const float* weight, int64_t M,
                                int K, float eps, int qmax, void* h, float* rstd, void* y, int8_t* xq, float* xs,
                                hipStream_t stream);
int64_t rmsnorm_grad_partial_rows(int64_t M, int K);
hipError_t launch_rmsnorm_grad(const void* grad, const void* h, int stream_f32, const float* rstd, const float* weight,
                               const void* grad_h, int64_t M, int K, int rot, void* dx, float* dweight, float* partial,
                               hipStream_t stream);
int64_t rope_grid(int64_t T, int heads, int head_dim, int pairs);
hipError_t launch_rope(const void* x, int64_t T, int heads, int head_dim, int64_t x_stride, const w4a8_rope* rope,
                       int inverse, void* out, int64_t out_stride, hipStream_t stream);
int64_t append_pages_per_seq(int64_t max_new, int page_tokens);
hipError_t launch_append(const w4a8_kv8& c, const int32_t* ctx_len, const int32_t* q_start, int64_t B, int64_t T,
                         int64_t max_new, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                         const void* q, int q_heads, int64_t q_stride, const w4a8_rope* rope, void* q_out,
                         int64_t out_stride, hipStream_t stream);
hipError_t launch_attention(const void* q, int q_heads, int64_t q_stride, const w4a8_kv8& c, const int32_t* kv_len,
                            const int32_t* q_start, int64_t B, int64_t T, int64_t max_new, int64_t max_kv, float scale,
                            int causal, int64_t window, void* out, int64_t out_stride, float* lse, float* workspace,
                            hipStream_t stream);
}  // namespace w4a8

namespace {

// Largest token, row and sequence counts: with at most 2^15 heads a product with them stays
// in 64 bits, and a launch of at most MAX_BLOCKS blocks of 256 threads in the grid limits.
constexpr int64_t MAX_TOKENS = int64_t(1) << 30;
constexpr int32_t MAX_HEADS = 1 << 15;
constexpr int64_t MAX_BLOCKS = (int64_t(1) << 24) - 1;
// 1024 threads a block at most in the norm kernels
constexpr int64_t MAX_NORM_BLOCKS = (int64_t(1) << 22) - 1;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int launched(hipError_t e) { return e == hipSuccess ? W4A8_OK : W4A8_ERR_HIP; }

int check_norm(int64_t M, int64_t K, int32_t stream_type) {
    if (M < 0 || K < 0) return W4A8_ERR_INVALID_ARG;
    if (K < W4A8_ROT_BLOCK || K % W4A8_ROT_BLOCK != 0) return W4A8_ERR_SHAPE;
    if (K > W4A8_NORM_MAX_K) return W4A8_ERR_UNSUPPORTED;
    if (M > MAX_NORM_BLOCKS) return W4A8_ERR_SHAPE;
    if (stream_type != W4A8_STREAM_BF16 && stream_type != W4A8_STREAM_F32) return W4A8_ERR_INVALID_ARG;
    return W4A8_OK;
}

// Dense heads, token stride in elements.
int check_heads(int64_t heads, int64_t head_dim, int64_t stride) {
    if (heads < 1 || head_dim < 1) return W4A8_ERR_INVALID_ARG;
    if (heads > MAX_HEADS) return W4A8_ERR_SHAPE;
    if (stride < heads * head_dim) return W4A8_ERR_SHAPE;
    if (stride % 8 != 0) return W4A8_ERR_ALIGN;
    return W4A8_OK;
}

int check_rope(const w4a8_rope* r, int64_t T, int32_t head_dim) {
    if (r->axes < 1 || r->axes > W4A8_ROPE_MAX_AXES) return W4A8_ERR_INVALID_ARG;
    if (r->interleaved != 0 && r->interleaved != 1) return W4A8_ERR_INVALID_ARG;
    if (r->rotary_dim < 16 || r->rotary_dim > head_dim || r->rotary_dim % 16 != 0) return W4A8_ERR_SHAPE;
    int64_t sum = 0;
    for (int i = 0; i < r->axes; ++i) {
        if (r->sections[i] < 0) return W4A8_ERR_INVALID_ARG;
        sum += r->sections[i];
    }
    if (sum != r->rotary_dim / 2) return W4A8_ERR_SHAPE;
    if (r->pos_stride < T) return W4A8_ERR_SHAPE;
    if (T > 0 && (!r->pos || !r->inv_freq)) return W4A8_ERR_INVALID_ARG;
    if (!aligned(r->pos, 4) || !aligned(r->inv_freq, 4)) return W4A8_ERR_ALIGN;
    return W4A8_OK;
}

int check_cache(const w4a8_kv8* c, int64_t B) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || (B != 0 && !c->table)) return W4A8_ERR_INVALID_ARG;
    if (c->heads < 1 || c->pages < 1 || c->table_stride < 1) return W4A8_ERR_INVALID_ARG;
    if (c->heads > MAX_HEADS || c->pages > INT32_MAX) return W4A8_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128) return W4A8_ERR_UNSUPPORTED;
    if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
        return W4A8_ERR_UNSUPPORTED;
    if ((int64_t)c->table_stride * c->page_tokens > MAX_TOKENS) return W4A8_ERR_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
        !aligned(c->table, 4))
        return W4A8_ERR_ALIGN;
    return W4A8_OK;
}

int check_batch(int64_t B, int64_t T, int64_t max_new) {
    if (B < 0 || T < 0 || max_new < 0) return W4A8_ERR_INVALID_ARG;
    if (B > MAX_TOKENS || T > MAX_TOKENS || max_new > MAX_TOKENS) return W4A8_ERR_SHAPE;
    return W4A8_OK;
}

// No sequence has more new tokens than there are rows.
int64_t bounded_new(int64_t T, int64_t max_new) { return max_new < T ? max_new : T; }

// The division of an attention's work (max_new <= T), or false if it is too large: its query rows, and the
// pairs of a row tile and a cache head that its sequences can have, are below the limit of a launch's
// blocks.  Rows are counted once, not as if every sequence had max_new of them.  The first three
// tests keep the plan's own products in 64 bits.
bool plan_of(int64_t B, int64_t T, int64_t max_new, int64_t max_kv, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
             w4a8::AttentionPlan& p) {
    const int64_t rows = B * max_new < T ? B * max_new : T, widest = (max_new * (q_heads / kv_heads) + 127) / 128;
    if (B > MAX_BLOCKS || rows * q_heads > MAX_BLOCKS || B * kv_heads * widest > MAX_BLOCKS) return false;
    p = w4a8::attention_plan(B, max_new, max_kv, q_heads, kv_heads, head_dim);
    return p.blocks <= MAX_BLOCKS && B * kv_heads * p.tiles <= MAX_BLOCKS;
}

}  // namespace

extern "C" {

int rmsnorm_quant_act(const void* x, const void* residual, int32_t stream_type, const float* weight, int64_t M,
                      int64_t K, float eps, int32_t rot_block, int32_t qmax, void* h, float* rstd, void* y, int8_t* xq,
                      float* xs, void* stream) {
    const int st = check_norm(M, K, stream_type);
    if (st) return st;
    if (!(eps > 0.0f) || !isfinite(eps)) return W4A8_ERR_INVALID_ARG;
    if (rot_block != W4A8_ROT_BLOCK || qmax < 1 || qmax > 127) return W4A8_ERR_UNSUPPORTED;
    if ((xq == nullptr) != (xs == nullptr) || (!xq && !y)) {
        if (M > 0) return W4A8_ERR_INVALID_ARG;
    }
    if (h && !residual) return W4A8_ERR_INVALID_ARG;
    if (!weight || (M > 0 && !x)) return W4A8_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(h, 16) || !aligned(rstd, 4) ||
        !aligned(y, 16) || !aligned(xq, 16) || !aligned(xs, 4))
        return W4A8_ERR_ALIGN;
    if (M == 0) return W4A8_OK;
    return launched(w4a8::launch_rmsnorm_quant(x, residual, stream_type == W4A8_STREAM_F32, weight, M, (int)K, eps, qmax,
                                               h, rstd, y, xq, xs, static_cast<hipStream_t>(stream)));
}

int64_t rmsnorm_grad_workspace(int64_t M, int64_t K) {
    if (check_norm(M, K, W4A8_STREAM_BF16)) return 0;
    return w4a8::rmsnorm_grad_partial_rows(M, (int)K) * K * (int64_t)sizeof(float);
}

int rmsnorm_grad(const void* grad, const void* h, int32_t stream_type, const float* rstd, const float* weight,
                 const void* grad_h, int64_t M, int64_t K, int32_t rot_block, void* dx, float* dweight, void* workspace,
                 int64_t workspace_bytes, void* stream) {
    const int st = check_norm(M, K, stream_type);
    if (st) return st;
    if (rot_block != W4A8_ROT_BLOCK && rot_block != 0) return W4A8_ERR_UNSUPPORTED;
    if (!weight || (M > 0 && (!grad || !h || !rstd || !dx))) return W4A8_ERR_INVALID_ARG;
    if (M > 0 && dweight && (!workspace || workspace_bytes < rmsnorm_grad_workspace(M, K))) return W4A8_ERR_INVALID_ARG;
    if (!aligned(grad, 16) || !aligned(h, 16) || !aligned(rstd, 4) || !aligned(weight, 16) || !aligned(grad_h, 16) ||
        !aligned(dx, 16) || !aligned(dweight, 16) || !aligned(workspace, 16))
        return W4A8_ERR_ALIGN;
    if (M == 0 && !dweight) return W4A8_OK;
    return launched(w4a8::launch_rmsnorm_grad(grad, h, stream_type == W4A8_STREAM_F32, rstd, weight, grad_h, M, (int)K,
                                              rot_block != 0, dx, dweight, static_cast<float*>(workspace),
                                              static_cast<hipStream_t>(stream)));
}

int rope_axes(const void* x, int64_t T, int32_t heads, int32_t head_dim, int64_t x_stride, const w4a8_rope* rope,
              int32_t inverse, void* out, int64_t out_stride, void* stream) {
    if (T < 0 || !rope || (inverse != 0 && inverse != 1)) return W4A8_ERR_INVALID_ARG;
    if (T > MAX_TOKENS) return W4A8_ERR_SHAPE;
    if (head_dim < 1) return W4A8_ERR_INVALID_ARG;
    if (head_dim % 16 != 0) return W4A8_ERR_SHAPE;
    if (head_dim > W4A8_ROPE_MAX_HEAD_DIM) return W4A8_ERR_UNSUPPORTED;
    int st = check_heads(heads, head_dim, x_stride);
    if (st) return st;
    if ((st = check_heads(heads, head_dim, out_stride))) return st;
    if ((st = check_rope(rope, T, head_dim))) return st;
    if (x == out && x_stride != out_stride) return W4A8_ERR_INVALID_ARG;
    if (T > 0 && (!x || !out)) return W4A8_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(out, 16)) return W4A8_ERR_ALIGN;
    if (T == 0) return W4A8_OK;
    if (w4a8::rope_grid(T, heads, head_dim, rope->rotary_dim / 2) > MAX_BLOCKS) return W4A8_ERR_SHAPE;
    return launched(w4a8::launch_rope(x, T, heads, head_dim, x_stride, rope, inverse, out, out_stride,
                                      static_cast<hipStream_t>(stream)));
}

int kv8_append(const w4a8_kv8* cache, const int32_t* ctx_len, const int32_t* q_start, int64_t B, int64_t T,
               int64_t max_new, const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q,
               int32_t q_heads, int64_t q_stride, const w4a8_rope* rope, void* q_out, int64_t out_stride,
               void* stream) {
    int st = check_cache(cache, B);
    if (st) return st;
    if ((st = check_batch(B, T, max_new))) return st;
    if ((st = check_heads(cache->heads, cache->head_dim, k_stride))) return st;
    if ((st = check_heads(cache->heads, cache->head_dim, v_stride))) return st;
    if ((q == nullptr) != (q_out == nullptr)) return W4A8_ERR_INVALID_ARG;
    if (q) {
        if ((st = check_heads(q_heads, cache->head_dim, q_stride))) return st;
        if ((st = check_heads(q_heads, cache->head_dim, out_stride))) return st;
        if (q == q_out && q_stride != out_stride) return W4A8_ERR_INVALID_ARG;
    }
    if (rope && (st = check_rope(rope, T, cache->head_dim))) return st;
    if (T > 0 && (!k || !v)) return W4A8_ERR_INVALID_ARG;
    if (B > 0 && (!ctx_len || !q_start)) return W4A8_ERR_INVALID_ARG;
    if (!aligned(ctx_len, 4) || !aligned(q_start, 4) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) ||
        !aligned(q_out, 16))
        return W4A8_ERR_ALIGN;
    if (T == 0) return W4A8_OK;
    max_new = bounded_new(T, max_new);
    const int64_t per_seq = w4a8::append_pages_per_seq(max_new, cache->page_tokens);
    const int64_t queries = q ? w4a8::rope_grid(T, q_heads, cache->head_dim, rope ? rope->rotary_dim / 2 : 0) : 0;
    if (per_seq > MAX_BLOCKS || B > MAX_BLOCKS || B * per_seq > MAX_BLOCKS ||
        B * per_seq * cache->heads * 2 + queries > MAX_BLOCKS)
        return W4A8_ERR_SHAPE;
    return launched(w4a8::launch_append(*cache, ctx_len, q_start, B, T, max_new, k, k_stride, v, v_stride, q, q_heads,
                                        q_stride, rope, q_out, out_stride, static_cast<hipStream_t>(stream)));
}

int64_t kv8_attention_workspace(int64_t B, int64_t T, int64_t max_new, int64_t max_kv, int32_t q_heads,
                                int32_t kv_heads, int32_t head_dim) {
    if (check_batch(B, T, max_new) || max_kv < 0 || max_kv > MAX_TOKENS || kv_heads < 1 || q_heads < kv_heads ||
        q_heads % kv_heads != 0 || q_heads > MAX_HEADS || (head_dim != 64 && head_dim != 128))
        return 0;
    max_new = bounded_new(T, max_new);
    w4a8::AttentionPlan p;
    if (B == 0 || max_new == 0 || !plan_of(B, T, max_new, max_kv, q_heads, kv_heads, head_dim, p)) return 0;
    return w4a8::attention_workspace(p, head_dim) * (int64_t)sizeof(float);
}

int kv8_attention(const void* q, int32_t q_heads, int64_t q_stride, const w4a8_kv8* cache, const int32_t* kv_len,
                  const int32_t* q_start, int64_t B, int64_t T, int64_t max_new, int64_t max_kv, float scale,
                  int32_t causal, int64_t window, void* out, int64_t out_stride, float* lse, void* workspace,
                  int64_t workspace_bytes, void* stream) {
    int st = check_cache(cache, B);
    if (st) return st;
    if ((st = check_batch(B, T, max_new))) return st;
    if (max_kv < 0 || window < 0 || (causal != 0 && causal != 1) || !(scale > 0.0f) || !isfinite(scale))
        return W4A8_ERR_INVALID_ARG;
    if (max_kv > MAX_TOKENS) return W4A8_ERR_SHAPE;
    if ((st = check_heads(q_heads, cache->head_dim, q_stride))) return st;
    if ((st = check_heads(q_heads, cache->head_dim, out_stride))) return st;
    if (q_heads % cache->heads != 0) return W4A8_ERR_SHAPE;
    if (T > 0 && (!q || !out)) return W4A8_ERR_INVALID_ARG;
    if (B > 0 && (!kv_len || !q_start)) return W4A8_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(kv_len, 4) || !aligned(q_start, 4) || !aligned(lse, 4) ||
        !aligned(workspace, 16))
        return W4A8_ERR_ALIGN;
    const int64_t need = kv8_attention_workspace(B, T, max_new, max_kv, q_heads, cache->heads, cache->head_dim);
    if (need > 0 && (!workspace || workspace_bytes < need)) return W4A8_ERR_INVALID_ARG;
    max_new = bounded_new(T, max_new);
    if (B == 0 || max_new == 0) return W4A8_OK;
    w4a8::AttentionPlan p;
    if (!plan_of(B, T, max_new, max_kv, q_heads, cache->heads, cache->head_dim, p)) return W4A8_ERR_SHAPE;
    return launched(w4a8::launch_attention(q, q_heads, q_stride, *cache, kv_len, q_start, B, T, max_new, max_kv, scale,
                                           causal, window, out, out_stride, lse, static_cast<float*>(workspace),
                                           static_cast<hipStream_t>(stream)));
}

int w4a8_block_abi_version(void) { return 1; }

}  // extern "C"
