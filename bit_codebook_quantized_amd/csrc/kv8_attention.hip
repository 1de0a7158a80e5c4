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
#include <type_traits>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/w4a8_block.h"
#include "kv8_plan.hpp"
#include "w4a8_device.hpp"

namespace w4a8 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int TILE = 64;             // keys of a step
constexpr int WAVES = 4;             // waves of a block: they share the rows and split the keys
constexpr int STEP = TILE * WAVES;   // keys of a block's step
constexpr float W_EXP = 15.0f;       // weights are kept times 2^15
constexpr int64_t DEAL_BLOCKS = 512;  // blocks that share the steps: two a CU

struct AttArgs {
    w4a8_kv8 c;
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    const int32_t* kv_len;
    const int32_t* q_start;
    int64_t q_stride, out_stride, T, max_new, window;
    float* part_o;        // dealt work, parts: [blocks * 2 * rows of a tile, head_dim], relative to
    float* part_ml;       // the part's own maximum; [.., 4]: that (log2 units), the two sums, unused
    int4* part_job;       // [blocks]: item (-1: nothing to join), head, last block, first slot
    float scale_log2;     // scale * log2(e)
    int q_heads, group, causal;
    int chunk_steps, chunks;   // many query rows: steps of a chunk of the context, most chunks
    int tiles, items;     // row tiles of a sequence with max_new tokens; of all sequences
};

// A value that every lane holds, into scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)uniform((int)v) | (uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32);
}

// The value itself, which the compiler cannot know to be the same in every turn of a loop: what
// is computed from it is computed anew in each turn instead of being held in registers.
__device__ __forceinline__ int anew(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

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

// The state of one query row, the same in its four lanes: maximum of the scores (log2 units),
// the sums (l for lse, lo divides the result), and log2 of the largest value scale that the row
// has seen.
struct RowState {
    float m, l, lo, lv;
};
__device__ __forceinline__ RowState fresh_row() { return RowState{-__builtin_inff(), 0.0f, 0.0f, -__builtin_inff()}; }

// The square root of a row's largest value scale: results take it twice, so that the scale may be
// subnormal, or so small that dividing it by the sum would make it so.
__device__ __forceinline__ float half_scale(const RowState& s) { return __builtin_amdgcn_exp2f(0.5f * s.lv); }

// Maximum and sum over the four lane groups of a row (lanes c, c + 16, c + 32, c + 48).
__device__ __forceinline__ float group_max(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t w = __float_as_uint(__builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
    const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return __builtin_fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float group_sum(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t w = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}

// What a lane knows of a tile: its 16 keys start at `key`, they are in one page.
struct TileInfo {
    float fk, fv;         // key scale times scale_log2, value scale
    float lfv, lvmax;     // log2 of fv (-inf below the smallest normal number), and the largest of the
                          // tile's pages (NaN left out)
    int key;
    bool present;         // the page exists
};
// With ONE_PAGE the whole tile is in one page.
template <bool ONE_PAGE>
__device__ __forceinline__ TileInfo tile_info(float k_scale, float v_scale, float scale_log2, int key, bool present) {
    TileInfo t;
    t.fk = k_scale * scale_log2;
    t.fv = v_scale;
    t.lfv = __builtin_amdgcn_logf(v_scale);
    t.lvmax = ONE_PAGE ? t.lfv : group_max(t.lfv);
    t.key = key;
    t.present = present;
    return t;
}
// Whether the tile needs no care: every page exists, has a positive value scale, and none of its
// value scales is below 2^-8 of the largest that the rows (lv) and the tile have met.  A weight then
// loses at most 2^-32 of the largest one to fp16's smallest step, in the sum as well.  And its key
// scale is below the rows' limit (score_limit).
template <bool ONE_PAGE>
__device__ __forceinline__ bool plain_tile(const TileInfo& t, float lv, float limit) {
    return __all(t.present & (t.lfv > (ONE_PAGE ? lv : __builtin_fmaxf(lv, t.lvmax)) - 8.0f) & (t.fk < limit));
}

// The factor of scores up to which none of this lane's query row can pass 2^12, whatever the codes
// are (0 for a row that is not finite).  From there on the exponent's bias in softmax_plain, which
// holds the maximum, would be off by more than 2^-11, and from 2^23 on by more than fp16 has room for.
// The sum of |q| comes out of a matrix product in every lane that holds a part of the row.
template <int N>
__device__ __forceinline__ float score_limit(const bf16x8 (&q)[N]) {
    const bf16x8 c = __builtin_bit_cast(bf16x8, make_uint4(0x43004300u, 0x43004300u, 0x43004300u, 0x43004300u));   // 128
    f32x4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        uint4 w = __builtin_bit_cast(uint4, q[i]);
        w.x &= 0x7FFF7FFFu; w.y &= 0x7FFF7FFFu; w.z &= 0x7FFF7FFFu; w.w &= 0x7FFF7FFFu;
        sum = mfma(c, __builtin_bit_cast(bf16x8, w), sum);
    }
    return sum[0] <= 3.402823466e38f ? 0x1p12f * __builtin_amdgcn_rcpf(sum[0]) : 0.0f;
}

struct Weights {
    f16x8 lo, hi;         // of this lane's tokens 0 .. 7 and 8 .. 15
};
__device__ __forceinline__ Weights weights_of(const uint32_t (&w)[8]) {
    return Weights{__builtin_bit_cast(f16x8, make_uint4(w[0], w[1], w[2], w[3])),
                   __builtin_bit_cast(f16x8, make_uint4(w[4], w[5], w[6], w[7]))};
}

// One tile's scores (acc, before scaling) to weights, the row's state, and the factor for its
// accumulated result; here where every row sees every key of a plain tile.  The value scale
// goes into the exponent, and (with one page) the sum of the weights is a matrix product with
// ones, both because the vector ALU is what this loop runs out of first.
template <bool ONE_PAGE>
__device__ __forceinline__ float softmax_plain(const f32x4 (&acc)[4], const TileInfo& t, bool want_lse, RowState& s,
                                               Weights& w) {
    float top = acc[0][0];
#pragma unroll
    for (int j = 1; j < 16; ++j) top = __builtin_fmaxf(top, acc[j >> 2][j & 3]);
    const float mn = __builtin_fmaxf(s.m, group_max(top * t.fk)), lvn = __builtin_fmaxf(s.lv, t.lvmax);
    const float r = t.lfv - lvn;
    const float alpha = __builtin_amdgcn_exp2f(s.m - mn), alpha_o = __builtin_amdgcn_exp2f((s.m - mn) + (s.lv - lvn));
    const float bias = (W_EXP - mn) + r;
    float p[16];
    uint32_t pw[8];
#pragma unroll
    for (int j = 0; j < 16; ++j) p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[j >> 2][j & 3], t.fk, bias));
#pragma unroll
    for (int j = 0; j < 8; ++j) pw[j] = pack_f16(p[2 * j], p[2 * j + 1]);
    w = weights_of(pw);
    // the sum of the weights without the value scale, as rounded; lse takes them as they were
    float sum = 0.0f;
    if constexpr (ONE_PAGE) {
        const f16x8 ones = {1, 1, 1, 1, 1, 1, 1, 1};
        f32x4 all = {0, 0, 0, 0};
        all = mfma(ones, w.lo, all);
        all = mfma(ones, w.hi, all);
        sum = all[0] * __builtin_amdgcn_exp2f(-r);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, pw[j]), f16x2{1, 1}, sum, false);
        sum = group_sum(sum * __builtin_amdgcn_exp2f(-r));
    }
    s.m = mn;
    s.lv = lvn;
    s.lo = __builtin_fmaf(s.lo, alpha, sum);
    if (want_lse) {
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) sum += p[j];
        sum = group_sum(sum * __builtin_amdgcn_exp2f(-r));
    }
    s.l = __builtin_fmaf(s.l, alpha, sum);
    return alpha_o;
}

// The same for any tile.  Few keys may count in one that is partly masked, so the sum that
// divides the result is taken of the weights as rounded (the rounding of a row with one key
// cancels, of few nearly), and the one for lse before; and a masked weight times a NaN scale
// must not reach the product, but one that is seen must, also where the weight has vanished.  A weight that the value scale brings below fp16's normal numbers
// counts in that sum as it was before the rounding, and so do all weights of a page whose scale
// leaves none above them: such keys add little or nothing to the product, but divide it like any other.
__device__ __forceinline__ float softmax_any(const f32x4 (&acc)[4], const TileInfo& t, int begin, int end, RowState& s,
                                             Weights& wt) {
    float x[16];
    float top = -__builtin_inff();
    bool any = false;
    const float lfv = __builtin_log2f(t.fv);       // of subnormal scales too
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int key = t.key + j;
        const bool seen = key < end && key >= begin && t.present;
        x[j] = seen ? acc[j >> 2][j & 3] * t.fk : -__builtin_inff();
        top = __builtin_fmaxf(top, x[j]);
        any |= seen;
    }
    const float lvn = group_max(__builtin_fmaxf(s.lv, any ? lfv : -__builtin_inff()));
    const float mn = __builtin_fmaxf(s.m, group_max(top));
    const float ref = mn > -__builtin_inff() ? mn : 0.0f;          // a row that has seen no key yet
    const float alpha = __builtin_amdgcn_exp2f(s.m - ref);
    const float alpha_o = s.lv == lvn ? alpha : alpha * __builtin_amdgcn_exp2f(s.lv - lvn);
    const float r = lfv > -__builtin_inff() ? __builtin_amdgcn_exp2f(lfv - lvn) : t.fv;
    float sum = 0.0f, rounded = 0.0f;
    uint32_t pw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        f16x2 w;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float p = __builtin_amdgcn_exp2f(x[2 * j + e] - ref + W_EXP);
            sum += p;
            const float scaled = x[2 * j + e] == -__builtin_inff() ? 0.0f : p * r;
            w[e] = (_Float16)scaled;
            rounded += scaled >= 0x1p-14f ? (float)w[e] : scaled;
        }
        pw[j] = __builtin_bit_cast(uint32_t, w);
    }
    wt = weights_of(pw);
    s.m = mn;
    s.lv = lvn;
    s.l = __builtin_fmaf(s.l, alpha, group_sum(sum));
    s.lo = __builtin_fmaf(s.lo, alpha, group_sum(any && r > 0x1p-29f ? rounded / r : sum));
    return alpha_o;
}

// The keys that rows row0 .. row0 + count - 1 of a sequence (count >= 1) see between them
// (from low to top) and all of them (from high to common).
struct Span {
    int low, top, high, common;
};
__device__ __forceinline__ Span span_of(const AttArgs& a, const Seq& s, int row0, int count) {
    const int first = s.pos0 + row0 / a.group, last = s.pos0 + (row0 + count - 1) / a.group;
    Span p;
    p.top = a.causal ? min(s.len, last + 1) : s.len;
    p.common = a.causal ? min(s.len, first + 1) : s.len;
    const int64_t lb = a.window > 0 ? (int64_t)first - a.window + 1 : 0, hb = a.window > 0 ? (int64_t)last - a.window + 1 : 0;
    p.low = lb > 0 ? (int)(lb < s.len ? lb : s.len) : 0;
    p.high = hb > 0 ? (int)(hb < s.len ? hb : s.len) : 0;
    return p;
}

// One query row: its place in q and out, and the keys it sees.  Lanes past a sequence's last row
// repeat it (and store nothing), so that they need no care.
struct Row {
    int token, head, begin, end;
};
__device__ __forceinline__ Row row_of(const AttArgs& a, const Seq& s, int kv_head, int row, int rows) {
    const int r = row < rows ? row : rows - 1;
    Row x;
    x.token = r / a.group;
    x.head = kv_head * a.group + r - x.token * a.group;
    const int pos = s.pos0 + x.token;
    x.end = a.causal && pos + 1 < s.len ? pos + 1 : s.len;
    x.begin = a.window > 0 && pos - a.window + 1 > 0 ? (int)(pos - a.window + 1) : 0;
    return x;
}

// Table entry of token `at` of a sequence (the index is bounded by its length first).
__device__ __forceinline__ int entry_at(const int32_t* table, int at, int len, int shift) {
    return table[(at < len ? at : len - 1) >> shift];
}
// The page that an entry names, -1 if it is not a page of the cache.
__device__ __forceinline__ int page_of(const AttArgs& a, int p) { return p >= 0 && p < a.c.pages ? p : -1; }

__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l) - W_EXP) * 0.69314718055994531f;
}

// Many query rows: from this many rows of a sequence on; waves of a block, each with one or two
// tiles of 16 rows.
constexpr int PROMPT_ROWS = 64, P_WAVES = 4;

// How the work of few query rows is dealt.  It is a list of steps: for every sequence, row tile (R rows) and
// head, the steps of S keys that its rows see.  The list is dealt to the blocks in equal
// contiguous shares, whatever the sequences' lengths are, so a block holds pieces of a few
// (row tile, head) pairs; a piece that is not all of one leaves its part in the workspace
// (a block has at most two such pieces: one that starts its share, one that ends it), and
// kv8_join_kernel adds the parts up.  Rows that see no key still have one (empty) step.
struct Item {            // one sequence's row tile
    Seq s;
    Span span;
    int row0, rows, steps;    // steps of one head, 0 if the tile has no rows
};
template <int R, int S>
__device__ __forceinline__ Item item_of(const AttArgs& a, int index) {
    Item x;
    x.s = seq_of(a, index / a.tiles);
    x.rows = x.s.n * a.group;
    x.row0 = (index % a.tiles) * R;
    x.steps = 0;
    x.span = Span{0, 0, 0, 0};
    if (x.row0 < x.rows) {
        x.span = span_of(a, x.s, x.row0, min(R, x.rows - x.row0));
        const int n = (x.span.top + S - 1) / S - x.span.low / S;
        x.steps = n > 0 ? n : 1;
    }
    return x;
}

// The item at the same index in every lane, in scalar registers.
template <int R, int S>
__device__ __forceinline__ Item one_item(const AttArgs& a, int index) {
    const Item v = item_of<R, S>(a, index);
    Item x;
    x.s = Seq{uniform(v.s.q0), uniform(v.s.n), uniform(v.s.len), uniform(v.s.pos0)};
    x.span = Span{uniform(v.span.low), uniform(v.span.top), uniform(v.span.high), uniform(v.span.common)};
    x.row0 = uniform(v.row0);
    x.rows = uniform(v.rows);
    x.steps = uniform(v.steps);
    return x;
}

__device__ __forceinline__ int64_t wave_prefix(int64_t v, int lane) {      // inclusive
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Steps of all items (whole wave).
template <int R, int S>
__device__ __forceinline__ int64_t total_steps(const AttArgs& a, int lane) {
    if (a.items == 1) return (int64_t)one_item<R, S>(a, 0).steps * a.c.heads;
    int64_t sum = 0;
    for (int i = 0; i < a.items; i += 64) {
        int64_t v = i + lane < a.items ? (int64_t)item_of<R, S>(a, i + lane).steps * a.c.heads : 0;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
        sum += v;
    }
    return uniform(sum);
}

// n / d for 0 <= n < 2^52, d > 0, the same in every lane: through fp64, put right by one where the quotient rounded up.
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
    const int64_t q = (int64_t)((double)n / (double)d);
    return uniform(q * d > n ? q - 1 : q);
}

// The list dealt to `blocks` blocks (at most one for each step): block i's share starts at
// from(i); the first `rest` shares are one step longer than the others.
struct Shares {
    int64_t blocks, each, rest;
    __device__ __forceinline__ int64_t from(int64_t i) const { return i * each + (i < rest ? i : rest); }
    __device__ __forceinline__ int64_t block_of(int64_t at) const {
        const int64_t longer = rest * (each + 1);
        return at < longer ? quotient(at, each + 1) : rest + quotient(at - longer, each);
    }
};
__device__ __forceinline__ Shares shares_of(int64_t total, int64_t blocks) {
    Shares s;
    s.blocks = blocks < total ? blocks : total;
    s.each = s.blocks > 0 ? quotient(total, s.blocks) : 0;
    s.rest = total - s.each * s.blocks;
    return s;
}

// The item that holds position `at` of the list (at < total), and where it starts.
template <int R, int S>
__device__ __forceinline__ int item_at(const AttArgs& a, int64_t at, int lane, int64_t& before) {
    before = 0;
    if (a.items == 1) return 0;
    int64_t sum = 0;
    for (int i = 0; i < a.items; i += 64) {
        const int64_t v = i + lane < a.items ? (int64_t)item_of<R, S>(a, i + lane).steps * a.c.heads : 0;
        const int64_t p = sum + wave_prefix(v, lane);
        const uint64_t past = __ballot(p > at);
        if (past != 0) {
            const int first = __ffsll((unsigned long long)past) - 1;
            before = uniform(__shfl(p - v, first));
            return uniform(i + first);
        }
        sum = __shfl(p, 63);
    }
    before = sum;
    return a.items;
}

// One block's share, piece by piece.
struct Piece {
    int index, head, step, steps;      // item, head, first step and how many
    int64_t slot;                      // part row of its first row, if it is not all of the item's steps
    bool whole;
};
template <int R, int S>
struct Walk {
    Shares deal;
    int64_t from, to, at, before;
    int index;

    // Whether this block has a share.
    __device__ __forceinline__ bool begin(const AttArgs& a, int lane) {
        deal = shares_of(total_steps<R, S>(a, lane), gridDim.x);
        if (blockIdx.x >= deal.blocks) return false;
        from = at = deal.from(blockIdx.x);
        to = deal.from(blockIdx.x + 1);
        index = item_at<R, S>(a, from, lane, before);
        return true;
    }
    // The next piece and its item.
    __device__ __forceinline__ bool next(const AttArgs& a, Piece& p, Item& x) {
        while (at < to && index < a.items) {
            x = one_item<R, S>(a, index);
            const int64_t size = (int64_t)x.steps * a.c.heads;
            if (at >= before + size) {         // this item is done (or has no rows)
                before += size;
                ++index;
                continue;
            }
            p.index = index;
            p.head = (int)quotient(at - before, x.steps);
            p.step = (int)((at - before) - (int64_t)p.head * x.steps);
            p.steps = (int)(to - at < x.steps - p.step ? to - at : x.steps - p.step);
            p.whole = p.steps == x.steps;
            p.slot = (2 * (int64_t)blockIdx.x + (at == from ? 0 : 1)) * R;
            // The piece that begins a row tile and head, and does not end it, names who joins the
            // parts: this block, up to the last block that has one.
            if (threadIdx.x == 0 && p.step == 0 && !p.whole)
                a.part_job[blockIdx.x] =
                    make_int4(index, p.head, (int)deal.block_of(at + x.steps - 1), at == from ? 0 : 1);
            at += p.steps;
            return true;
        }
        return false;
    }
    // Between pieces the state lies in LDS, a copy a wave, and not in registers.
    __device__ __forceinline__ void keep(Walk& lds) const {
        lds = *this;
        wave_lds_sync();
    }
};

template <int R, int S>
__device__ __forceinline__ bool next_piece(const AttArgs& a, Walk<R, S>& lds, Piece& p, Item& x) {
    Walk<R, S> w;
    w.deal = Shares{uniform(lds.deal.blocks), uniform(lds.deal.each), uniform(lds.deal.rest)};
    w.from = uniform(lds.from);
    w.to = uniform(lds.to);
    w.at = uniform(lds.at);
    w.before = uniform(lds.before);
    w.index = uniform(lds.index);
    const bool more = w.next(a, p, x);
    w.keep(lds);
    return more;
}

// Without dealing: block i takes all of one (row tile, head) pair, heads fastest, and the last
// row tiles of a sequence first (causal rows see more the later they are).
template <int R, int S>
__device__ __forceinline__ bool own_item(const AttArgs& a, Piece& p, Item& x) {
    const int i = blockIdx.x / a.c.heads;
    p.head = blockIdx.x % a.c.heads;
    p.index = i / a.tiles * a.tiles + a.tiles - 1 - i % a.tiles;
    x = one_item<R, S>(a, p.index);
    p.step = 0;
    p.steps = x.steps;
    p.slot = 0;
    p.whole = true;
    return x.steps > 0;
}

// A wave loads its tile straight into registers in the order of the matrix operands: the
// values of a tile while its scores are made, the keys of the next one while its weights are
// used.  The W waves take the step's W tiles and are joined through LDS.
// Bound by memory where the cache is long: 16 sequences of 2 k to 32 k tokens, 8 cache heads of
// 128: 109 us and 6 for the join, 4.9 TB/s of codes (with lse and without; a window of 1024: 21 us);
// loading the values a step ahead as well was 3 % slower.  By latency where it is short: 1000 tokens of
// one sequence 11.5 us, 300 tokens 7.9 us.  5 tokens each over up to 8 k: 51 us, over a window
// of 1024 28 us.
template <int D, bool ONE_PAGE, bool DEAL, int W>
__global__ __launch_bounds__(64 * W, 2) void kv8_attention_kernel(AttArgs a) {
    constexpr int NK = D / 64;       // 16-byte key loads a lane and sub-tile
    constexpr int NV = D / 16;       // value column tiles
    constexpr int R = 16;            // rows of a block
    constexpr int STEP = TILE * W;   // keys of a step
    // the waves' results: O^T [wave][D][16 + 1], maxima and sums
    __shared__ float so[W][D][16 + 1];
    __shared__ float sm[W][16], sl[W][16], slo[W][16];

    __shared__ Walk<R, STEP> walks[DEAL ? W : 1];
    const int wave = uniform((int)threadIdx.x >> 6);
    Piece piece;
    Item x;
    if constexpr (DEAL) {
        if (threadIdx.x == 0) a.part_job[blockIdx.x] = make_int4(-1, 0, 0, 0);
        Walk<R, STEP> walk;
        if (!walk.begin(a, threadIdx.x & 63) || !walk.next(a, piece, x)) return;
        walk.keep(walks[wave]);
    } else if (!own_item<R, STEP>(a, piece, x)) {
        return;
    }
    const int shift = 31 - __clz(a.c.page_tokens), in_page = a.c.page_tokens - 1;
    const bool want_lse = a.lse != nullptr;

    do {
        const int tid = DEAL ? anew(threadIdx.x) : threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
        const int head = piece.head;
        const Seq& s = x.s;
        const Span& span = x.span;
        const int rows = x.rows, row0 = x.row0;
        const int32_t* const table = a.c.table + (int64_t)(piece.index / a.tiles) * a.c.table_stride;
        const int first = (span.low / STEP + piece.step) * STEP;
        const int k0 = first + wave * TILE, k1 = min(span.top, first + piece.steps * STEP);

        const Row row = row_of(a, s, head, row0 + c, rows);
        bf16x8 qf[2 * NK];
        {
            const uint16_t* src = a.q + (s.q0 + row.token) * a.q_stride + (int64_t)row.head * D + 16 * g;
#pragma unroll
            for (int i = 0; i < 2 * NK; ++i)
                qf[i] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(src + 64 * (i >> 1) + 8 * (i & 1)));
        }
        RowState st = fresh_row();
        f32x4 o[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) o[i] = f32x4{0, 0, 0, 0};

        // lane (c, g): keys from row c of a sub-tile (tokens 16 (c / 4) + 4 j + c % 4), 16 codes
        // of every 64; values of tokens 16 g .. 16 g + 15.  Page numbers are fetched a step
        // before what they point at, and first looked at there (a look at once would wait for
        // the loads before them).
        uint4 kw[4 * NK];
        int entry_k = 0, entry_v = 0, pk = 0, pv = 0;
        auto pages = [&](int kt) {
            entry_k = entry_at(table, ONE_PAGE ? uniform(kt) : kt + 16 * (c >> 2), s.len, shift);
            if constexpr (!ONE_PAGE) entry_v = entry_at(table, kt + 16 * g, s.len, shift);
        };
        auto load_keys = [&](int kt) {
            pk = page_of(a, ONE_PAGE ? uniform(entry_k) : entry_k);
            pv = ONE_PAGE ? pk : page_of(a, entry_v);
            const int8_t* kp = a.c.k + ((((int64_t)(pk < 0 ? 0 : pk) * a.c.heads + head) << shift) +
                                        ((kt + 16 * (c >> 2)) & in_page) + (c & 3)) * D + 16 * g;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < NK; ++i) kw[j * NK + i] = *reinterpret_cast<const uint4*>(kp + 4 * j * D + 64 * i);
        };
        if (k0 < k1) {
            pages(k0);
            load_keys(k0);
        }
        float limit = 0.0f;
        for (int kt = k0; kt < k1; kt += STEP) {
            const int64_t vpage = (int64_t)(pv < 0 ? 0 : pv) * a.c.heads + head;
            const int8_t* vp = a.c.v + ((vpage * D) << shift) + ((int64_t)c << shift) + ((kt + 16 * g) & in_page);
            const float ks = a.c.k_scale[vpage], vs = a.c.v_scale[vpage];
            const bool present = pv >= 0;
            const bool more = kt + STEP < k1;
            if (more) pages(kt + STEP);
            uint4 vw[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) vw[i] = *reinterpret_cast<const uint4*>(vp + ((int64_t)(16 * i) << shift));

            f32x4 acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[j] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < NK; ++i) {
                    const uint4 w = kw[j * NK + i];
                    acc[j] = mfma(widen(w.x, w.y), qf[2 * i], acc[j]);
                    acc[j] = mfma(widen(w.z, w.w), qf[2 * i + 1], acc[j]);
                }
            }
            if (more) load_keys(kt + STEP);
            if (kt == k0) limit = score_limit(qf);      // here, where the first loads are under way
            const TileInfo t = tile_info<ONE_PAGE>(ks, vs, a.scale_log2, kt + 16 * g, present);
            const bool plain = kt + TILE <= span.common && kt >= span.high && plain_tile<ONE_PAGE>(t, st.lv, limit);
            Weights w;
            const float alpha = plain ? softmax_plain<ONE_PAGE>(acc, t, want_lse, st, w)
                                      : softmax_any(acc, t, row.begin, row.end, st, w);
            if (__any(alpha != 1.0f)) {
#pragma unroll
                for (int i = 0; i < NV; ++i) o[i] *= alpha;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                o[i] = mfma(widen_f16(vw[i].x, vw[i].y), w.lo, o[i]);
                o[i] = mfma(widen_f16(vw[i].z, vw[i].w), w.hi, o[i]);
            }
        }
        const float vhalf = half_scale(st);
        if (g == 0) { sm[wave][c] = st.m; sl[wave][c] = st.l; slo[wave][c] = st.lo; }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) so[wave][16 * i + 4 * g + e][c] = o[i][e] * vhalf * vhalf;
        __syncthreads();

        // join the waves: 4 W threads a row
        const int r = tid / (4 * W), d0 = tid % (4 * W), mine = row0 + r;
        if (mine < rows) {
            float mt = sm[0][r];
#pragma unroll
            for (int w = 1; w < W; ++w) mt = __builtin_fmaxf(mt, sm[w][r]);
            const float ref = mt > -__builtin_inff() ? mt : 0.0f;
            float f[W], lt = 0.0f, lot = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                f[w] = __builtin_amdgcn_exp2f(sm[w][r] - ref);
                lt += sl[w][r] * f[w];
                lot += slo[w][r] * f[w];
            }
            const int out_token = mine / a.group, out_head = head * a.group + mine % a.group;
            const int64_t t = s.q0 + out_token, rid = t * a.q_heads + out_head;
            const int64_t slot = piece.slot + r;
            const float inv = lt == 0.0f ? 0.0f : 1.0f / lot;      // a row that sees no key: 0
#pragma unroll
            for (int i = 0; i < D / (4 * W); ++i) {
                const int d = d0 + 4 * W * i;
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) v = __builtin_fmaf(so[w][d][r], f[w], v);
                if (!DEAL || piece.whole) a.out[t * a.out_stride + (int64_t)out_head * D + d] = f32_to_bf16(lt == 0.0f ? 0.0f : v * inv);
                else a.part_o[slot * D + d] = v;
            }
            if (d0 == 0) {
                if (DEAL && !piece.whole) *reinterpret_cast<float4*>(a.part_ml + slot * 4) = make_float4(mt, lt, lot, 0.0f);
                else if (a.lse) a.lse[rid] = lse_of(mt, lt);
            }
        }
        __syncthreads();       // before the next results
    } while (DEAL && next_piece(a, walks[wave], piece, x));
}

// First part row of a (row tile, head) pair's chunk (many query rows, R a block).
template <int R>
__device__ __forceinline__ int64_t part_slot(const AttArgs& a, int index, int head, int chunk) {
    return (((int64_t)index * a.c.heads + head) * a.chunks + chunk) * R;
}

// Joins the parts of one (row tile, head) pair, 16 rows a block: the W waves take parts in turn,
// four at a time (their loads are what this kernel waits for), with a running maximum, then
// join through LDS; of many query rows, with few parts each, they take rows in turn instead.  A lane has 4 columns of every 64 / (D / 4)-th row.  Few query rows: the pair that block blockIdx.x of the main launch began.  Many: the
// pair's chunks.
template <int D, bool MANY, int R, int W>
__global__ __launch_bounds__(64 * W) void kv8_join_kernel(AttArgs a) {
    constexpr int LANES = D / 4, AT_ONCE = 64 / LANES, NR = 16 / AT_ONCE;
    constexpr int SHARE = MANY ? 1 : W;      // waves that share a row's parts
    __shared__ __attribute__((aligned(16))) float so[SHARE][16][D];
    __shared__ float sm[SHARE][16], sl[SHARE][16], slo[SHARE][16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int sub = lane / LANES, col = 4 * (lane % LANES);
    int head, count, row0, parts;
    int64_t q0, slot0, slot1;       // slots of the first part and of the second; the others follow it
    constexpr int64_t NEXT = MANY ? R : 2 * R;
    const int sub0 = blockIdx.x % (R / 16) * 16;
    if constexpr (MANY) {
        const int pair = blockIdx.x / (R / 16);
        head = pair % a.c.heads;
        const Item x = one_item<R, TILE>(a, pair / a.c.heads);
        parts = min(a.chunks, (x.steps + a.chunk_steps - 1) / a.chunk_steps);
        row0 = x.row0 + sub0;
        count = min(16, x.rows - row0);
        if (parts < 2 || count <= 0) return;
        q0 = x.s.q0;
        slot0 = part_slot<R>(a, pair / a.c.heads, head, 0) + sub0;
        slot1 = slot0 + NEXT;
    } else {
        const int block = blockIdx.x / (R / 16);
        const int4 job = a.part_job[block];
        if (job.x < 0) return;
        const Item x = one_item<R, STEP>(a, uniform(job.x));
        head = job.y;
        row0 = x.row0 + sub0;
        count = min(16, x.rows - row0);
        if (count <= 0) return;
        q0 = x.s.q0;
        parts = job.z - block + 1;
        slot0 = (2 * (int64_t)block + job.w) * R + sub0;
        slot1 = 2 * ((int64_t)block + 1) * R + sub0;
    }

    auto finish = [&](int r, int d, f32x4 y, float mt, float lt, float lot) {
        const int64_t t = q0 + (row0 + r) / a.group;
        const int qh = head * a.group + (row0 + r) % a.group;
        const float inv = 1.0f / lot;
        *reinterpret_cast<uint2*>(a.out + t * a.out_stride + (int64_t)qh * D + d) =
            lt == 0.0f ? make_uint2(0, 0) : make_uint2(f32x2_to_bf16x2(y[0] * inv, y[1] * inv), f32x2_to_bf16x2(y[2] * inv, y[3] * inv));
        if (a.lse && d == 0) a.lse[t * a.q_heads + qh] = lse_of(mt, lt);
    };
#pragma unroll 1
    for (int j = MANY ? wave : 0; j < NR; j += MANY ? W : 1) {
        const int r = AT_ONCE * j + sub;
        if (AT_ONCE * j >= count) break;
        const int rr = r < count ? r : count - 1;
        f32x4 v = {0, 0, 0, 0};
        float m = -__builtin_inff(), l = 0.0f, lo = 0.0f;
        for (int i = MANY ? 0 : wave; i < parts; i += 4 * SHARE) {
            float4 ml[4];
            f32x4 p[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int part = i + u * SHARE < parts ? i + u * SHARE : i;
                const int64_t slot = (part == 0 ? slot0 : slot1 + (part - 1) * NEXT) + rr;
                ml[u] = *reinterpret_cast<const float4*>(a.part_ml + slot * 4);
                p[u] = *reinterpret_cast<const f32x4*>(a.part_o + slot * D + col);
            }
            float mn = m;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (i + u * SHARE >= parts) ml[u].x = -__builtin_inff();       // counted already
                mn = __builtin_fmaxf(mn, ml[u].x);
            }
            const float ref = mn > -__builtin_inff() ? mn : 0.0f, old = __builtin_amdgcn_exp2f(m - ref);
            m = mn;
            l *= old;
            lo *= old;
            v *= old;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float f = __builtin_amdgcn_exp2f(ml[u].x - ref);
                l = __builtin_fmaf(ml[u].y, f, l);
                lo = __builtin_fmaf(ml[u].z, f, lo);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(p[u][e], f, v[e]);
            }
        }
        if (r >= count) continue;
        if constexpr (MANY) {
            finish(r, col, v, m, l, lo);
        } else {
            *reinterpret_cast<f32x4*>(&so[wave][r][col]) = v;
            if (col == 0) { sm[wave][r] = m; sl[wave][r] = l; slo[wave][r] = lo; }
        }
    }
    if constexpr (MANY) return;
    __syncthreads();
    for (int i = tid; i < count * LANES; i += 64 * W) {
        const int r = i / LANES, d = 4 * (i % LANES);
        float mt = sm[0][r];
#pragma unroll
        for (int w = 1; w < SHARE; ++w) mt = __builtin_fmaxf(mt, sm[w][r]);
        const float ref = mt > -__builtin_inff() ? mt : 0.0f;
        float lt = 0.0f, lot = 0.0f;
        f32x4 y = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < SHARE; ++w) {
            const float f = __builtin_amdgcn_exp2f(sm[w][r] - ref);
            lt += sl[w][r] * f;
            lot += slo[w][r] * f;
            const f32x4 p = *reinterpret_cast<const f32x4*>(&so[w][r][d]);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(p[e], f, y[e]);
        }
        finish(r, d, y, mt, lt, lot);
    }
}

// Place of 16-byte piece p of row r of an LDS tile whose rows have W pieces (8 or 16): the
// pieces are exchanged among the rows that share banks (256 bytes), so that the 16 lanes that
// read one piece of 16 consecutive rows each meet every bank once.
template <int W>
__device__ __forceinline__ int lds_piece(int r, int p) {
    static_assert(W == 8 || W == 16, "128- or 256-byte rows");
    return W * r + (p ^ (W == 16 ? r & 15 : (r >> 1) & 7));
}

// Many query rows: a block has 64 or 128 of them, 16 or 32 a wave, and all its waves walk the
// same keys.  A tile is widened once a block on its way into LDS (two tiles in turn: the next one
// is loaded while this one is used, one barrier a tile).  A key lies at row 16 j + 4 a + b of the
// tile for key 16 a + 4 j + b, so that the 16 rows of a sub-tile follow each other; tokens
// 16 g + 8 e .. + 7 of a value column are its piece 4 e + g.  Two blocks share a CU and are not
// in step, so one's matrix work meets the other's vector work (one block of 256 rows, whose
// waves pass the barrier together, was 5 % faster on 4096 of 16384 tokens and 15 to 30 %
// slower on prompts of 2000).  Reads are issued four ahead of the products that use them, which
// the compiler does not do itself.  With 128 rows (4096 of 16384 tokens, 32 heads of 128: 993 us, 969
// TFLOP/s) a wave issues 380 vector instructions a tile, 68 of them matrix products: by the counters
// vector issue takes 65 % of a SIMD's time and the matrix units 42 %, LDS reads 40 % of a CU's (a
// quarter of that bank conflicts); matrix and vector work overlap, but do not hide each other.  With 64
// rows (prompts of 2000 and 125, 16 heads of 64) it is 15 other vector instructions for each matrix one:
// vector issue takes 78 %, matrix units 18 %, and the last causal rows are the longest chain of
// steps: with HALVES = 2 waves 4 to 7 take every second tile, beside the others, and the two results are
// added in LDS at the end.  2048 of 2048 tokens 66 to 70 us with lse and without, a window of 1024 50,
// not causal 84.
template <int D, bool ONE_PAGE, bool SPLIT, bool LSE, int P_QT, int HALVES = 1>
__global__ __launch_bounds__(64 * P_WAVES * HALVES, 2) void kv8_prompt_kernel(AttArgs a) {
    static_assert(HALVES == 1 || (HALVES == 2 && !SPLIT && P_QT == 1), "halves of a whole context");
    constexpr int NS = D / 32, NV = D / 16;
    constexpr int P_ROWS = 16 * P_QT * P_WAVES;
    constexpr int AHEAD = 4;         // fragments read before the product that uses the first
    constexpr int CHUNKS = TILE * D / 16;                   // 16-code pieces of a tile's keys, or values
    constexpr int STRIDE = HALVES * TILE;                   // from a wave's tile to its next one
    __shared__ __attribute__((aligned(16))) uint16_t sk_all[HALVES][2][TILE * D];
    __shared__ __attribute__((aligned(16))) uint16_t sv_all[HALVES][2][D * TILE];

    const int half = HALVES == 1 ? 0 : uniform((int)threadIdx.x / (64 * P_WAVES));
    const int tid = threadIdx.x % (64 * P_WAVES), wave = uniform(tid >> 6);
    auto& sk = sk_all[half];
    auto& sv = sv_all[half];
    const int shift = 31 - __clz(a.c.page_tokens), in_page = a.c.page_tokens - 1;
    // heads fastest, then the context's chunks, then the row tiles of a sequence, the last ones
    // first (causal rows see more the later they are)
    int id = blockIdx.x;
    const int head = id % a.c.heads;
    id /= a.c.heads;
    const int chunk = SPLIT ? id % a.chunks : 0;
    if (SPLIT) id /= a.chunks;
    const int index = id / a.tiles * a.tiles + a.tiles - 1 - id % a.tiles;
    const Item x = one_item<P_ROWS, TILE>(a, index);
    const int step = SPLIT ? chunk * a.chunk_steps : 0, left = x.steps - step;
    const int steps = SPLIT && chunk < a.chunks - 1 ? min(left, a.chunk_steps) : left;
    if (steps <= 0) return;
    const bool all = !SPLIT || steps == x.steps;
    const int lane = tid & 63, c = lane & 15, g = lane >> 4;
    const Seq& s = x.s;
    const Span& span = x.span;
    const int rows = x.rows, row0 = x.row0;
    const int32_t* const table = a.c.table + (int64_t)(index / a.tiles) * a.c.table_stride;
    const int k0 = (span.low / TILE + step) * TILE, k1 = min(span.top, k0 + steps * TILE);

    // this wave's rows
    const int wrow0 = row0 + 16 * P_QT * wave;
    const bool idle = wrow0 >= rows;
    const Span wspan = span_of(a, s, idle ? row0 : wrow0, idle ? 1 : min(16 * P_QT, rows - wrow0));
    Row row[P_QT];
    bf16x8 qf[P_QT][NS];
#pragma unroll
    for (int t = 0; t < P_QT; ++t) {
        row[t] = row_of(a, s, head, wrow0 + 16 * t + c, rows);
        const uint16_t* src = a.q + (s.q0 + row[t].token) * a.q_stride + (int64_t)row[t].head * D + 8 * g;
#pragma unroll
        for (int i = 0; i < NS; ++i) qf[t][i] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(src + 32 * i));
    }
    RowState st[P_QT];
    f32x4 o[P_QT][NV];
#pragma unroll
    for (int t = 0; t < P_QT; ++t) {
        st[t] = fresh_row();
#pragma unroll
        for (int i = 0; i < NV; ++i) o[t][i] = f32x4{0, 0, 0, 0};
    }

    // This thread's pieces of the staged tile: 16 codes of a key, and 16 of a value column.  A
    // wave has 16 tokens' keys, so one page's; and their values, where a tile has several pages
    // (with one page neighbouring threads read a column's 64 tokens instead).
    constexpr int NP = CHUNKS / (64 * P_WAVES);
    static_assert(NP * 64 * P_WAVES == CHUNKS, "whole pieces a thread");
    static_assert(P_WAVES * 16 == TILE, "16 tokens a wave");
    auto piece_key = [&](int p) { return 16 * wave + (lane + 64 * p) / (D / 16); };
    auto piece_dim = [&](int p) { return 16 * (lane % (D / 16)); };
    auto piece_col = [&](int p) { return ONE_PAGE ? (tid + 64 * P_WAVES * p) >> 2 : lane + 64 * p; };
    const int stok = 16 * (ONE_PAGE ? tid & 3 : wave);
    uint4 kw[NP], vw[NP];
    // Page numbers are fetched a tile before what they point at, and first looked at there (a
    // look at once would wait for the tile's loads before them): of the staged pieces, and (for
    // the scales) of this lane's 16 tokens.
    int entry = 0, scale_entry = 0;
    auto pages = [&](int kt) {
        entry = entry_at(table, ONE_PAGE ? kt : kt + 16 * wave, s.len, shift);
        if constexpr (!ONE_PAGE) scale_entry = entry_at(table, kt + 16 * g, s.len, shift);
    };
    float ks = 0.0f, vs = 0.0f;        // of the tile that is loaded
    bool present = false;
    auto load = [&](int kt) {
        const int pp = page_of(a, uniform(entry)), ps = ONE_PAGE ? pp : page_of(a, scale_entry);
        const int64_t page = (((int64_t)(pp < 0 ? 0 : pp) * a.c.heads + head) << shift) * D;
        const int8_t* keys = a.c.k + page;
        const int8_t* values = a.c.v + page;
#pragma unroll
        for (int p = 0; p < NP; ++p)
            kw[p] = *reinterpret_cast<const uint4*>(keys + (uint32_t)(((kt + piece_key(p)) & in_page) * D + piece_dim(p)));
#pragma unroll
        for (int p = 0; p < NP; ++p)
            vw[p] = *reinterpret_cast<const uint4*>(values + (uint32_t)((piece_col(p) << shift) + ((kt + stok) & in_page)));
        // byte offsets in 32 bits: a page and head has 2048 codes or more, so the card holds fewer than 2^28
        const uint32_t at = 4u * ((uint32_t)(ps < 0 ? 0 : ps) * (uint32_t)a.c.heads + (uint32_t)head);
        ks = *reinterpret_cast<const float*>(reinterpret_cast<const char*>(a.c.k_scale) + at);
        vs = *reinterpret_cast<const float*>(reinterpret_cast<const char*>(a.c.v_scale) + at);
        present = ps >= 0;
    };
    auto store = [&](int kbuf, int vbuf) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int key = piece_key(p), row = 16 * ((key >> 2) & 3) + 4 * (key >> 4) + (key & 3), at = piece_dim(p) / 8;
            uint4* k = reinterpret_cast<uint4*>(sk[kbuf]);
            k[lds_piece<D / 8>(row, at)] = __builtin_bit_cast(uint4, widen(kw[p].x, kw[p].y));
            k[lds_piece<D / 8>(row, at + 1)] = __builtin_bit_cast(uint4, widen(kw[p].z, kw[p].w));
            uint4* v = reinterpret_cast<uint4*>(sv[vbuf]);
            v[lds_piece<8>(piece_col(p), stok / 16)] = __builtin_bit_cast(uint4, widen_f16(vw[p].x, vw[p].y));
            v[lds_piece<8>(piece_col(p), stok / 16 + 4)] = __builtin_bit_cast(uint4, widen_f16(vw[p].z, vw[p].w));
        }
    };

    // The weights of a tile that this wave has not yet used.
    Weights w[P_QT];
    float alpha[P_QT];
    auto use_weights = [&](int vbuf) {
#pragma unroll
        for (int t = 0; t < P_QT; ++t)
            if (__any(alpha[t] != 1.0f)) {
#pragma unroll
                for (int i = 0; i < NV; ++i) o[t][i] *= alpha[t];
            }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const f16x8 v = __builtin_bit_cast(
                    f16x8, reinterpret_cast<const uint4*>(sv[vbuf])[lds_piece<8>(c, 4 * e + g) + 16 * 8 * i]);
#pragma unroll
                for (int t = 0; t < P_QT; ++t) o[t][i] = mfma(v, e ? w[t].hi : w[t].lo, o[t][i]);
            }
        __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
        for (int i = 0; i < 2 * NV - AHEAD; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, P_QT, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, AHEAD * P_QT, 0);
    };

    const int first = k0 + TILE * half;
    float limit = 0.0f;
    if (first < k1) {
        pages(first);
        load(first);
        pages(first + STRIDE);
        limit = score_limit(qf[0]);        // here, where the first tile is on its way
#pragma unroll
        for (int t = 1; t < P_QT; ++t) limit = __builtin_fminf(limit, score_limit(qf[t]));
        store(0, 0);
    }
    // The queries have arrived: a wait for them inside the loop would wait for the tile that is
    // being fetched as well.
    __builtin_amdgcn_s_waitcnt(0x0F70);      // vmcnt(0)
    int kbuf = 0, vbuf = 0;             // of this tile
    for (int kt = first; kt < k1 + TILE * half; kt += STRIDE) {     // as many steps in both halves
        const int vnext = vbuf ^ 1;
        __syncthreads();
        const bool more = kt + STRIDE < k1;
        const TileInfo info = tile_info<ONE_PAGE>(ks, vs, a.scale_log2, kt + 16 * g, present);
        if (more) {
            load(kt + STRIDE);
            pages(kt + 2 * STRIDE);
        }
        if (!idle && kt < wspan.top && kt + TILE > wspan.low) {
            f32x4 acc[P_QT][4];
#pragma unroll
            for (int i = 0; i < NS; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (i == 0)
#pragma unroll
                        for (int t = 0; t < P_QT; ++t) acc[t][j] = f32x4{0, 0, 0, 0};
                    const bf16x8 k = __builtin_bit_cast(
                        bf16x8, reinterpret_cast<const uint4*>(sk[kbuf])[lds_piece<D / 8>(c, 4 * i + g) + 16 * (D / 8) * j]);
#pragma unroll
                    for (int t = 0; t < P_QT; ++t) acc[t][j] = mfma(k, qf[t][i], acc[t][j]);
                }
            }
            __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 1);
#pragma unroll
            for (int i = 0; i < 4 * NS - AHEAD; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, P_QT, 1);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 1);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, AHEAD * P_QT, 1);
            const bool plain = kt + TILE <= wspan.common && kt >= wspan.high &&
                               plain_tile<ONE_PAGE>(info, P_QT == 1 ? st[0].lv : __builtin_fmaxf(st[0].lv, st[P_QT - 1].lv), limit);
            if (plain) {
#pragma unroll
                for (int t = 0; t < P_QT; ++t) alpha[t] = softmax_plain<ONE_PAGE>(acc[t], info, LSE, st[t], w[t]);
            } else {
#pragma unroll
                for (int t = 0; t < P_QT; ++t)
                    alpha[t] = softmax_any(acc[t], info, row[t].begin, row[t].end, st[t], w[t]);
            }
            use_weights(vbuf);
        }
        if (more) store(kbuf ^ 1, vnext);
        kbuf ^= 1;
        vbuf = vnext;
    }

    if constexpr (HALVES == 2) {
        // the second half's results go to the same lanes of the first
        f32x4* so = reinterpret_cast<f32x4*>(sk_all);
        float4* sml = reinterpret_cast<float4*>(sv_all);
        const float vhalf = half_scale(st[0]);
        __syncthreads();
        if (half == 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i) so[64 * P_WAVES * i + tid] = o[0][i] * vhalf * vhalf;
            sml[tid] = make_float4(st[0].m, st[0].l, st[0].lo, 0.0f);
        }
        __syncthreads();
        if (half == 1) return;
        const float4 other = sml[tid];
        const float top = __builtin_fmaxf(st[0].m, other.x), ref = top > -__builtin_inff() ? top : 0.0f;
        const float f0 = __builtin_amdgcn_exp2f(st[0].m - ref), f1 = __builtin_amdgcn_exp2f(other.x - ref);
        st[0].l = st[0].l * f0 + other.y * f1;
        st[0].lo = st[0].lo * f0 + other.z * f1;
        st[0].m = top;
        st[0].lv = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) o[0][i] = o[0][i] * vhalf * vhalf * f0 + so[64 * P_WAVES * i + tid] * f1;
    }

    // lane (c, g) holds columns 16 i + 4 g .. + 3 of its rows
#pragma unroll
    for (int t = 0; t < P_QT; ++t) {
        const float l = st[t].l, lo = st[t].lo, vhalf = half_scale(st[t]);
        if (wrow0 + 16 * t + c >= rows) continue;
        const Row mine = row_of(a, s, head, wrow0 + 16 * t + c, rows);
        const int64_t tok = s.q0 + mine.token;
        if (all) {
            const float inv = l == 0.0f ? 0.0f : vhalf / lo;
            uint16_t* dst = a.out + tok * a.out_stride + (int64_t)mine.head * D + 4 * g;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const f32x4 v = o[t][i] * vhalf * inv;
                *reinterpret_cast<uint2*>(dst + 16 * i) =
                    l == 0.0f ? make_uint2(0, 0) : make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
            }
            if (LSE && g == 0) a.lse[tok * a.q_heads + mine.head] = lse_of(st[t].m, l);
        } else {
            const int64_t slot = part_slot<P_ROWS>(a, index, head, chunk) + 16 * (P_QT * wave + t) + c;
            float* dst = a.part_o + slot * D + 4 * g;
#pragma unroll
            for (int i = 0; i < NV; ++i) *reinterpret_cast<f32x4*>(dst + 16 * i) = o[t][i] * vhalf * vhalf;
            if (g == 0) *reinterpret_cast<float4*>(a.part_ml + slot * 4) = make_float4(st[t].m, l, lo, 0.0f);
        }
    }
}

template <int N>
using Size = std::integral_constant<int, N>;

}  // namespace

// Blocks of a launch.  Times of two sides are of one build each; the present one is within 3 % of them.
// Few rows, short contexts, few of them: a block of 8 waves for each pair, no parts (1 x 1000
// tokens, 8 cache heads: 11.3 us against 11.9 and a launch more; 1 x 2048: 16.4 against 12.5;
// 16 x up to 2048: 17.7 against 20.8; 16 x up to 4096: 28.1 against 27.5).
// Few rows otherwise (a step is 256 keys): one for each (row tile, head), or 512 (two a CU, as many as fit
// at once) that share all steps equally and whose parts are then joined.  Dealing costs a second
// launch and pays where pairs would leave blocks idle, by three steps; lengths are uneven as a
// rule, so contexts of eight steps are dealt however many pairs there are (16 x up to 32 k
// tokens: 181 us in fixed splits, 115 dealt; 256 x up to 400: 57 us dealt, 34 us a block each).
// Many rows (a step is 64 keys), 32 query heads over 8 cache heads of 128 in these times: from 64
// rows a sequence on (4 x 16 tokens of 8192: 27 us, in 16-row tiles 38; 40 rows would gain over
// 8192, 45 and 35, and lose over 500, 9.1 and 12.3).  128 rows a block where that gives two
// blocks a CU, four in contexts below 32 steps, or where few new tokens look back on a long
// context; else 64, whose steps are shorter but reuse what they read half as often.  With 128 and
// 64 rows: 500 of 500 tokens 20.7 and 13.3 us, 1024 of 1024 36 and 26, 2 x 1000 of 1000 35 and 27,
// 2048 of 2048 66 and 68, 2500 of 2500 80 and 94, 16 x 500 of 500 41 and 48, 4 x 128 of 8192
// 66 and 75, 8 x 24 of 8192 46.8 and 45.8.  One block for each pair, or, where pairs are less than
// two a CU, for each chunk of a pair's context: about 1024 (2048 with 64 rows) in all, no less
// than six steps a chunk (64 rows over 16 steps or fewer are not cut, 4 x 64 of 1024: 19.6 us,
// cut 22.2; 130 of 1500: 20.1, cut 13.3).  Where pairs of 64 rows are up to twice what fits at
// once with eight waves (two blocks a CU at 64 columns, one at 128), eight waves take every second
// tile each: the longest chain of steps is half as long (without and with: prompts of 2000 and
// 125, 16 heads of 64, 48 and 42 us; 1024 of 1024 28 and 27, 500 of 500 15.1 and 13.3; with more
// pairs, 2 x 1000 of 1000, 27 and 31, 5 x 500 of 500 21 and 29).
AttentionPlan attention_plan(int64_t B, int64_t max_new, int64_t max_kv, int q_heads, int kv_heads, int head_dim) {
    const int group = q_heads / kv_heads;
    const int64_t query_rows = max_new * group;
    AttentionPlan p{};
    p.prompt = query_rows >= PROMPT_ROWS;
    auto pairs = [&](int rows) { return B * kv_heads * ((query_rows + rows - 1) / rows); };
    if (p.prompt) {
        const int64_t steps = std::max<int64_t>(1, (max_kv + TILE - 1) / TILE);
        const bool looks_back = query_rows >= 128 && 8 * max_new <= max_kv && pairs(128) * steps >= 4 * DEAL_BLOCKS;
        p.rows = pairs(128) >= (steps < 32 ? 2 : 1) * DEAL_BLOCKS || looks_back ? 128 : 64;
        p.tiles = (query_rows + p.rows - 1) / p.rows;
        const int64_t base = pairs(p.rows), blocks = (p.rows == 128 ? 2 : 4) * DEAL_BLOCKS;
        const int64_t chunk = std::max<int64_t>(6, (base * steps + blocks - 1) / blocks);
        p.parts = base < DEAL_BLOCKS && (p.rows == 64 ? steps > 16 : 2 * steps > 3 * chunk);
        // a context longer than max_kv is still walked: its last chunk is the longest
        p.chunks = p.parts ? (int)((steps + chunk - 1) / chunk) : 1;
        p.chunk_steps = (int)chunk;
        p.halves = p.rows == 64 && !p.parts && base <= (head_dim == 64 ? 2 : 1) * DEAL_BLOCKS;
        p.blocks = base * p.chunks;
        p.join_blocks = p.parts ? base * (p.rows / 16) : 0;
        p.part_rows = p.parts ? base * p.chunks * p.rows : 0;
        return p;
    }
    p.rows = 16;
    p.tiles = (query_rows + 15) / 16;
    const int64_t base = pairs(16);
    const int64_t steps = std::max<int64_t>(1, (max_kv + STEP - 1) / STEP);
    p.wide = base <= 256 && max_kv <= (base < 64 ? 1024 : 2048);
    if (p.wide) {
        p.blocks = base;
        return p;
    }
    p.parts = steps >= 8 || steps * std::max<int64_t>(0, DEAL_BLOCKS - base) >= 3 * DEAL_BLOCKS;
    p.blocks = p.parts ? std::min<int64_t>(DEAL_BLOCKS, base * steps) : base;
    p.join_blocks = p.parts ? p.blocks * (p.rows / 16) : 0;
    p.part_rows = p.parts ? p.blocks * 2 * p.rows : 0;
    return p;
}

// Floats of workspace.
int64_t attention_workspace(const AttentionPlan& p, int head_dim) {
    return p.parts ? p.part_rows * (head_dim + 4) + (p.prompt ? 0 : 4 * p.blocks) : 0;
}

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
    const AttentionPlan p = attention_plan(B, max_new, max_kv, q_heads, c.heads, c.head_dim);
    a.part_o = workspace;
    a.part_ml = workspace + p.part_rows * c.head_dim;
    a.part_job = reinterpret_cast<int4*>(a.part_ml + p.part_rows * 4);
    a.chunk_steps = p.chunk_steps;
    a.chunks = p.chunks;
    a.tiles = (int)p.tiles;
    a.items = (int)(B * a.tiles);
    const dim3 grid((unsigned)p.blocks), join((unsigned)p.join_blocks);
    // pages of at least a tile: its page number and scales are one for all lanes
    auto with_sizes = [&](auto&& go) {
        const bool one = c.page_tokens >= TILE;
        if (c.head_dim == 64) { if (one) go(Size<64>{}, std::true_type{}); else go(Size<64>{}, std::false_type{}); }
        else { if (one) go(Size<128>{}, std::true_type{}); else go(Size<128>{}, std::false_type{}); }
    };
    auto with_flag = [](bool flag, auto&& go) { if (flag) go(std::true_type{}); else go(std::false_type{}); };
    with_sizes([&](auto d, auto one) {
        constexpr int D = decltype(d)::value;
        constexpr bool ONE = decltype(one)::value;
        with_flag(p.parts, [&](auto parts) {
            constexpr bool PARTS = decltype(parts)::value;
            if (p.prompt) {
                with_flag(lse != nullptr, [&](auto want) {
                    constexpr bool LSE = decltype(want)::value;
                    if (p.rows == 128) hipLaunchKernelGGL((kv8_prompt_kernel<D, ONE, PARTS, LSE, 2>), grid, dim3(64 * P_WAVES), 0, stream, a);
                    else if (p.halves) hipLaunchKernelGGL((kv8_prompt_kernel<D, ONE, false, LSE, 1, 2>), grid, dim3(128 * P_WAVES), 0, stream, a);
                    else hipLaunchKernelGGL((kv8_prompt_kernel<D, ONE, PARTS, LSE, 1>), grid, dim3(64 * P_WAVES), 0, stream, a);
                });
            } else if (p.wide) {
                hipLaunchKernelGGL((kv8_attention_kernel<D, ONE, false, 2 * WAVES>), grid, dim3(128 * WAVES), 0, stream, a);
            } else {
                hipLaunchKernelGGL((kv8_attention_kernel<D, ONE, PARTS, WAVES>), grid, dim3(64 * WAVES), 0, stream, a);
            }
        });
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.parts) return e;
    with_sizes([&](auto d, auto) {
        constexpr int D = decltype(d)::value;
        if (p.rows == 128) hipLaunchKernelGGL((kv8_join_kernel<D, true, 128, 4>), join, dim3(256), 0, stream, a);
        else if (p.rows == 64) hipLaunchKernelGGL((kv8_join_kernel<D, true, 64, 4>), join, dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((kv8_join_kernel<D, false, 16, 8>), join, dim3(512), 0, stream, a);
    });
    return hipGetLastError();
}

}  // namespace w4a8
