// kv8_attention: softmax attention over the 8-bit paged cache (include/w4a8_block.h).
//
// One pass over the keys with a running maximum and sum for each query row.  Everything is
// computed transposed, S^T = K Q^T and O^T = V^T P^T, with 16x16x32 bf16 matrix
// instructions: a lane then holds one query row (column lane % 16) in S^T, in the weights
// and in O^T alike, so its running maximum and the rescaling are one number a lane, and
// the weights go from the first product to the second without leaving their lane:
//   - a tile is 64 keys.  Lane (c, g) = (lane % 16, lane / 16).  Sub-tile j of S^T takes
//     as row r the key 16 (r / 4) + 4 j + r % 4, so lane group g ends with the 16
//     consecutive keys 16 g .. 16 g + 15 of its query row;
//   - the second product wants, from lane group g, weights and values of its own 16
//     tokens: exactly those.  The values lie transposed in the cache, so 16 tokens of one
//     value column are one 16-byte load.
// The scores are bf16 products: queries are bf16 and codes are exact in it (|code| <= 127
// needs 7 bits).  The second product is in fp16, where codes are exact too and a weight
// keeps 11 bits instead of 8.  Its range is kept by normalising: a weight is stored as
// 2^15 w r <= 2^15, with w = exp(score - running maximum) and r the value scale of its page
// over the largest one met so far, so all weights above 2^-29 are normal numbers.
// The rows of a tile are (token, query head) pairs of one cache head, so a group of query
// heads shares the keys that it reads.
#include <algorithm>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/w4a8_block.h"
#include "w4a8_device.hpp"

namespace w4a8 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int TILE = 64;             // keys of a step
constexpr int ROWS = 16;             // query rows of a block
constexpr int WAVES = 4;             // waves of a block: they share the rows and split the keys
constexpr int STEP = TILE * WAVES;   // keys of a block's step
constexpr float W_EXP = 15.0f;       // weights are kept times 2^15

struct AttArgs {
    w4a8_kv8 c;
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    const int32_t* kv_len;
    const int32_t* q_start;
    int64_t q_stride, out_stride, T, max_new, window;
    float* part_o;        // [T * q_heads, splits, head_dim], of this split's own maximum
    float* part_ml;       // [T * q_heads, splits, 4]: maximum (log2 units), the two sums, unused
    float scale_log2;     // scale * log2(e)
    int q_heads, group, causal;
    int tiles;            // row tiles of a sequence with max_new tokens
    int splits, chunk;    // keys of a split (a multiple of STEP); the last one takes the rest
};

// The query rows of sequence b: how many new tokens, where they start, how long the cache is.
struct Seq {
    int64_t q0;
    int n, len, pos0;     // pos0: position of the first new token (may be negative)
};
__device__ __forceinline__ Seq seq_of(const AttArgs& a, int64_t b) {
    int64_t q0 = a.q_start[b], q1 = a.q_start[b + 1];
    q0 = q0 < 0 ? 0 : q0;
    q1 = q1 > a.T ? a.T : q1;
    const int64_t n = q1 > q0 ? q1 - q0 : 0;
    const int64_t most = (int64_t)a.c.table_stride * a.c.page_tokens;
    int64_t len = a.kv_len[b];
    len = len < 0 ? 0 : len > most ? most : len;
    Seq s;
    s.q0 = q0;
    s.len = (int)len;
    s.pos0 = (int)(len - n);
    s.n = (int)(n < a.max_new ? n : a.max_new);
    return s;
}

// 8 codes to bf16, exactly: through fp32, whose upper half is the bf16 value.
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = i < 2 ? lo >> (16 * i) : hi >> (16 * (i - 2));
        const float a = (float)(int8_t)x, b = (float)(int8_t)(x >> 8);
        w[i] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
    }
    return __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
}

// 8 codes to fp16, exactly: 0x6400 | u is 1024 + u for a byte u = code + 128.
__device__ __forceinline__ f16x8 widen_f16(uint32_t lo, uint32_t hi) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = (i < 2 ? lo : hi) ^ 0x80808080u;
        const uint32_t x = __builtin_amdgcn_perm(0x64646464u, u, i & 1 ? 0x04030402u : 0x04010400u);
        w[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, x) - (f16x2){1152, 1152});
    }
    return __builtin_bit_cast(f16x8, make_uint4(w[0], w[1], w[2], w[3]));
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Page that holds tokens at .. of sequence b, or -1 (the token index is bounded first).
__device__ __forceinline__ int64_t page_at(const AttArgs& a, const int32_t* table, int token, int len, int shift) {
    const int t = token < len ? token : len - 1;
    const int64_t p = table[t >> shift];
    return p >= 0 && p < a.c.pages ? p : -1;
}

template <int D>
__global__ __launch_bounds__(64 * WAVES) void kv8_attention_kernel(AttArgs a) {
    constexpr int NK = D / 64;       // 16-byte key loads a lane and sub-tile
    constexpr int NV = D / 16;       // value columns tiles
    // the waves' results, joined at the end: O^T [wave][D][16 + 1], maxima and sums
    __shared__ float so[WAVES][D][ROWS + 1];
    __shared__ float sm[WAVES][ROWS], sl[WAVES][ROWS], slo[WAVES][ROWS];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, g = lane >> 4;
    int id = blockIdx.x;                               // split fastest, then head, row tile, sequence
    const int split = id % a.splits;
    id /= a.splits;
    const int head = id % a.c.heads;
    id /= a.c.heads;
    const int64_t b = id / a.tiles;
    const int tile_rows = id % a.tiles;
    const Seq s = seq_of(a, b);
    const int rows = s.n * a.group;
    const int row0 = tile_rows * ROWS;
    if (row0 >= rows) return;
    const int shift = 31 - __clz(a.c.page_tokens);
    const int32_t* const table = a.c.table + b * a.c.table_stride;

    // this lane's query row
    const int row = row0 + c, rr = row < rows ? row : rows - 1;
    const int token = rr / a.group, qh = head * a.group + rr % a.group;
    const int pos = s.pos0 + token;
    int end = a.causal && pos + 1 < s.len ? pos + 1 : s.len;          // keys below it are seen
    int begin = a.window > 0 && pos - a.window + 1 > 0 ? (int)(pos - a.window + 1) : 0;
    if (row >= rows) end = 0;
    // what the block's rows see between them, and what all of them see
    const int last_token = (min(row0 + ROWS, rows) - 1) / a.group, first_token = row0 / a.group;
    const int top_end = a.causal ? min(s.len, s.pos0 + last_token + 1) : s.len;
    const int low_end = a.causal ? min(s.len, s.pos0 + first_token + 1) : s.len;
    const int64_t lb = a.window > 0 ? (int64_t)s.pos0 + first_token - a.window + 1 : 0;
    const int64_t hb = a.window > 0 ? (int64_t)s.pos0 + last_token - a.window + 1 : 0;
    const int low_begin = lb > 0 ? (int)lb : 0;
    const int top_begin = hb > 0 ? (int)(hb < s.len ? hb : s.len) : 0;
    const bool whole = row0 + ROWS <= rows;

    const int k_first = split * a.chunk;
    const int k0 = max(k_first, low_begin / STEP * STEP);
    const int k1 = split == a.splits - 1 ? top_end : min(top_end, k_first + a.chunk);

    bf16x8 qf[2 * NK];
    {
        const uint16_t* src = a.q + (s.q0 + token) * a.q_stride + (int64_t)qh * D;
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                qf[2 * i + e] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(src + 64 * i + 16 * g + 8 * e));
    }

    float m = -__builtin_inff(), l = 0.0f;
    float lo = 0.0f;                 // the sum that divides the result (l is the one for lse)
    float vtop = 0.0f;               // largest value scale that the row has seen
    f32x4 o[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) o[i] = f32x4{0, 0, 0, 0};

    for (int kt = k0 + wave * TILE; kt < k1; kt += STEP) {
        // keys: lane c loads rows of the page of tokens 16 (c / 4) .., values and scales: of 16 g ..
        const int64_t pk = page_at(a, table, kt + 16 * (c >> 2), s.len, shift);
        const int64_t pv = page_at(a, table, kt + 16 * g, s.len, shift);
        const int in_page = (1 << shift) - 1;
        const int8_t* kp = a.c.k + (((pk < 0 ? 0 : pk) * a.c.heads + head) << shift) * D +
                           (int64_t)(((kt + 16 * (c >> 2)) & in_page) + (c & 3)) * D + 16 * g;
        const int64_t vbase = (pv < 0 ? 0 : pv) * a.c.heads + head;
        const int8_t* vp = a.c.v + ((vbase * D) << shift) + ((int64_t)c << shift) + ((kt + 16 * g) & in_page);
        const float fk = a.c.k_scale[vbase] * a.scale_log2, fv = a.c.v_scale[vbase];

        f32x4 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                const uint4 w = *reinterpret_cast<const uint4*>(kp + 4 * j * D + 64 * i);
                acc[j] = mfma(widen(w.x, w.y), qf[2 * i], acc[j]);
                acc[j] = mfma(widen(w.z, w.w), qf[2 * i + 1], acc[j]);
            }
        }
        float x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = acc[j >> 2][j & 3] * fk;
        const bool masked = !whole || kt + TILE > low_end || kt < top_begin || __any(pv < 0);
        if (masked) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int key = kt + 16 * g + j;
                x[j] = key < end && key >= begin && pv >= 0 ? x[j] : -__builtin_inff();
            }
        }
        float top = x[0];
#pragma unroll
        for (int j = 1; j < 16; ++j) top = __builtin_fmaxf(top, x[j]);
        // the largest value scale of the pages that the row has seen (a NaN one is left to its
        // own weights)
        float vn = __builtin_fmaxf(vtop, masked && top == -__builtin_inff() ? 0.0f : fv);
        top = __builtin_fmaxf(top, __shfl_xor(top, 16));
        top = __builtin_fmaxf(top, __shfl_xor(top, 32));
        vn = __builtin_fmaxf(vn, __shfl_xor(vn, 16));
        vn = __builtin_fmaxf(vn, __shfl_xor(vn, 32));
        const float mn = __builtin_fmaxf(m, top);
        const float ref = mn > -__builtin_inff() ? mn : 0.0f;      // a row that has seen no key yet
        const float alpha = __builtin_amdgcn_exp2f(m - ref);
        const float inv_top = vn > 0.0f ? 1.0f / vn : 0.0f;
        const float alpha_o = alpha * (vtop * inv_top), r = fv * inv_top;
        m = mn;
        vtop = vn;
#pragma unroll
        for (int i = 0; i < NV; ++i) o[i] *= alpha_o;
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = __builtin_amdgcn_exp2f(x[j] - ref + W_EXP);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) sum += x[j];
        l = l * alpha + sum;
        uint32_t pw[8];
        if (masked) {
            // few keys may count here: their sum is taken of the weights as rounded, so that the
            // roundings of a row with one key cancel, of few nearly; and a masked weight
            // times a NaN scale must not reach the product
            float rounded = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f16x2 w;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    w[e] = (_Float16)(x[2 * j + e] == 0.0f ? 0.0f : x[2 * j + e] * r);
                    rounded += (float)w[e];
                }
                pw[j] = __builtin_bit_cast(uint32_t, w);
            }
            lo = lo * alpha + (r > 0.0f ? rounded / r : sum);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                pw[j] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)(x[2 * j] * r), (_Float16)(x[2 * j + 1] * r)});
            lo = lo * alpha + sum;
        }
        const f16x8 pf0 = __builtin_bit_cast(f16x8, make_uint4(pw[0], pw[1], pw[2], pw[3]));
        const f16x8 pf1 = __builtin_bit_cast(f16x8, make_uint4(pw[4], pw[5], pw[6], pw[7]));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint4 w = *reinterpret_cast<const uint4*>(vp + ((int64_t)(16 * i) << shift));
            o[i] = mfma(widen_f16(w.x, w.y), pf0, o[i]);
            o[i] = mfma(widen_f16(w.z, w.w), pf1, o[i]);
        }
    }
    // a lane's l covers its own 16 keys of each tile
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    lo += __shfl_xor(lo, 16);
    lo += __shfl_xor(lo, 32);

    if (g == 0) { sm[wave][c] = m; sl[wave][c] = l; slo[wave][c] = lo; }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) so[wave][16 * i + 4 * g + e][c] = o[i][e] * vtop;
    __syncthreads();

    // join the waves: thread (r, d ..) takes row r
    const int r = tid >> 4, d0 = tid & 15;     // 16 rows x 16 threads
    if (row0 + r >= rows) return;
    float mt = sm[0][r];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) mt = __builtin_fmaxf(mt, sm[w][r]);
    const float ref = mt > -__builtin_inff() ? mt : 0.0f;
    float f[WAVES], lt = 0.0f, lot = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        f[w] = __builtin_amdgcn_exp2f(sm[w][r] - ref);
        lt += sl[w][r] * f[w];
        lot += slo[w][r] * f[w];
    }
    const int out_token = (row0 + r) / a.group, out_head = head * a.group + (row0 + r) % a.group;
    const int64_t t = s.q0 + out_token;
    const float inv = lt == 0.0f ? 0.0f : 1.0f / lot;      // a row that sees no key: 0
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        const int d = d0 + 16 * i;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) v = __builtin_fmaf(so[w][d][r], f[w], v);
        if (a.splits == 1) a.out[t * a.out_stride + (int64_t)out_head * D + d] = f32_to_bf16(lt == 0.0f ? 0.0f : v * inv);
        else a.part_o[((t * a.q_heads + out_head) * a.splits + split) * D + d] = v;
    }
    if (d0 == 0) {
        const int64_t id = t * a.q_heads + out_head;
        if (a.splits > 1) {
            float* ml = a.part_ml + (id * a.splits + split) * 4;
            ml[0] = mt;
            ml[1] = lt;
            ml[2] = lot;
        } else if (a.lse) {
            a.lse[id] = lt == 0.0f ? -__builtin_inff() : (mt + __builtin_log2f(lt) - W_EXP) * 0.69314718055994531f;
        }
    }
}

// Joins the splits of one query row: 64 threads a row, D / 64 columns each.
template <int D>
__global__ __launch_bounds__(64) void kv8_join_kernel(AttArgs a) {
    int bid = blockIdx.x;
    const int lane = threadIdx.x, head = bid % a.c.heads;
    bid /= a.c.heads;
    const int most = (int)a.max_new * a.group, row = bid % most;
    const int64_t b = bid / most;
    const Seq s = seq_of(a, b);
    if (row >= s.n * a.group) return;
    const int64_t t = s.q0 + row / a.group;
    const int qh = head * a.group + row % a.group;
    const int64_t id = t * a.q_heads + qh;
    const float* ml = a.part_ml + id * a.splits * 4;
    const float* po = a.part_o + id * a.splits * D;
    float mt = -__builtin_inff();
    for (int i = 0; i < a.splits; ++i) mt = __builtin_fmaxf(mt, ml[4 * i]);
    const float ref = mt > -__builtin_inff() ? mt : 0.0f;
    float lt = 0.0f, lot = 0.0f, v[D / 64];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) v[j] = 0.0f;
    for (int i = 0; i < a.splits; ++i) {
        const float f = __builtin_amdgcn_exp2f(ml[4 * i] - ref);
        lt += ml[4 * i + 1] * f;
        lot += ml[4 * i + 2] * f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) v[j] = __builtin_fmaf(po[(int64_t)i * D + lane + 64 * j], f, v[j]);
    }
    const float inv = 1.0f / lot;
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
        a.out[t * a.out_stride + (int64_t)qh * D + lane + 64 * j] = f32_to_bf16(lt == 0.0f ? 0.0f : v[j] * inv);
    if (a.lse && lane == 0) a.lse[id] = lt == 0.0f ? -__builtin_inff() : (mt + __builtin_log2f(lt) - W_EXP) * 0.69314718055994531f;
}

int64_t row_tiles(int64_t max_new, int group) { return (max_new * group + ROWS - 1) / ROWS; }

}  // namespace

// How the context is divided: enough splits for about 8 blocks a CU, none shorter than two
// steps, at most 64.
int attention_splits(int64_t B, int64_t max_new, int64_t max_kv, int q_heads, int kv_heads) {
    const int64_t base = std::max<int64_t>(1, B * kv_heads * row_tiles(max_new, q_heads / kv_heads));
    const int64_t want = (2048 + base - 1) / base, most = std::max<int64_t>(1, max_kv / (2 * STEP));
    return (int)std::min<int64_t>(64, std::min(want, most));
}

// Blocks of the main launch and of the join.
int64_t attention_blocks(int64_t B, int64_t max_new, int64_t max_kv, int q_heads, int kv_heads) {
    return B * row_tiles(max_new, q_heads / kv_heads) * kv_heads *
           attention_splits(B, max_new, max_kv, q_heads, kv_heads);
}
int64_t attention_join_blocks(int64_t B, int64_t max_new, int q_heads) { return B * max_new * q_heads; }

hipError_t launch_attention(const void* q, int q_heads, int64_t q_stride, const w4a8_kv8& c, const int32_t* kv_len,
                            const int32_t* q_start, int64_t B, int64_t T, int64_t max_new, int64_t max_kv, float scale,
                            int causal, int64_t window, void* out, int64_t out_stride, float* lse, float* workspace,
                            hipStream_t stream) {
    (void)hipGetLastError();   // clear a stale error so the check below is about this launch
    AttArgs a{};
    a.c = c;
    a.q = static_cast<const uint16_t*>(q);
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.kv_len = kv_len; a.q_start = q_start;
    a.q_stride = q_stride; a.out_stride = out_stride; a.T = T; a.max_new = max_new; a.window = window;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.q_heads = q_heads; a.group = q_heads / c.heads; a.causal = causal;
    a.splits = attention_splits(B, max_new, max_kv, q_heads, c.heads);
    a.chunk = (int)((max_kv + a.splits - 1) / a.splits + STEP - 1) / STEP * STEP;
    a.part_o = workspace;
    a.part_ml = workspace + T * q_heads * a.splits * c.head_dim;
    a.tiles = (int)row_tiles(max_new, a.group);
    const dim3 grid((unsigned)attention_blocks(B, max_new, max_kv, q_heads, c.heads));
    if (c.head_dim == 64) hipLaunchKernelGGL(kv8_attention_kernel<64>, grid, dim3(64 * WAVES), 0, stream, a);
    else hipLaunchKernelGGL(kv8_attention_kernel<128>, grid, dim3(64 * WAVES), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const dim3 jgrid((unsigned)attention_join_blocks(B, max_new, q_heads));
    if (c.head_dim == 64) hipLaunchKernelGGL(kv8_join_kernel<64>, jgrid, dim3(64), 0, stream, a);
    else hipLaunchKernelGGL(kv8_join_kernel<128>, jgrid, dim3(64), 0, stream, a);
    return hipGetLastError();
}

}  // namespace w4a8
