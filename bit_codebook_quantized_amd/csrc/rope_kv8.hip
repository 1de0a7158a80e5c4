// rope_axes and kv8_append: rotary positions with several axes, and the append of new keys
// and values to the 8-bit paged cache (include/w4a8_block.h states the formulas).
//
// Angles: pos * inv_freq in revolutions, as one fp64 product (24-bit frequency times 31-bit
// position, 1 / 2 pi to 53 bits), reduced to (-1/2, 1/2] by subtracting its rounding, and
// only then narrowed to fp32: within 2^-25 of a revolution for positions up to 2^28, where an
// fp32 product would lose a bit for every doubling of the position.
#include <algorithm>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/w4a8_block.h"
#include "w4a8_device.hpp"

namespace w4a8 {
namespace {

// The kernel's view of w4a8_rope (pos NULL: no rotation).
struct RopeArgs {
    const int32_t* pos;
    int64_t pos_stride;
    const float* inv_freq;
    int32_t pairs;                        // rotary_dim / 2
    int32_t end[W4A8_ROPE_MAX_AXES];      // pairs below end[a] (and not below end[a - 1]) are of axis a
    int32_t interleaved;
    float sign;                           // -1 turns the other way
};

// cos and sin of pair p's angle for token t.
__device__ __forceinline__ float2 rope_turn(const RopeArgs& r, int64_t t, int p) {
    int a = 0;
#pragma unroll
    for (int i = 0; i < W4A8_ROPE_MAX_AXES - 1; ++i) a += p >= r.end[i] ? 1 : 0;
    const double f = (double)r.inv_freq[p] * 0.15915494309189533577;   // revolutions a position
    double rev = (double)r.pos[a * r.pos_stride + t] * f;
    rev -= __builtin_rint(rev);
    float s, c;
    sincospif(2.0f * (float)rev, &s, &c);
    return make_float2(c, s * r.sign);
}

// A head is head_dim / 16 pieces of 16 elements in two halves of 8: a piece of the rotated
// part holds 8 pairs, (a, b) = (lo[i], hi[i]) for split pairs and the neighbours within
// lo then hi for interleaved ones; pieces past rotary_dim hold 16 neighbours.
struct Piece {
    int lo, hi;    // element offsets in the head
    int pair;      // first of its 8 pairs, -1 past the rotated part
};
__device__ __forceinline__ Piece piece_of(const RopeArgs& r, int c) {
    const int turned = r.pairs >> 3;
    if (c < turned && !r.interleaved) return Piece{8 * c, r.pairs + 8 * c, 8 * c};
    return Piece{16 * c, 16 * c + 8, c < turned ? 8 * c : -1};
}

__device__ __forceinline__ void widen8(const uint4 a, float (&v)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 narrow8(const float (&v)[8]) {
    return make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                      f32x2_to_bf16x2(v[6], v[7]));
}

// Each output is two rounded products and one rounded sum.
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
    const float x = a * c - b * s;
    b = b * c + a * s;
    a = x;
}
// One pair i (of 8) of a piece.
__device__ __forceinline__ void turn_in_piece(float (&lo)[8], float (&hi)[8], int i, bool interleaved, float2 cs) {
    if (!interleaved) turn_pair(lo[i], hi[i], cs.x, cs.y);
    else if (i < 4) turn_pair(lo[2 * i], lo[2 * i + 1], cs.x, cs.y);
    else turn_pair(hi[2 * i - 8], hi[2 * i - 7], cs.x, cs.y);
}

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_LDS_PAIRS = ROPE_THREADS;    // cos/sin entries of a block: tokens a block times pairs

struct RopeRun {    // one tensor to rotate
    const uint16_t* x;
    uint16_t* out;
    int64_t T, x_stride, out_stride;
    int heads, head_dim;
    int tokens_per_block, heads_per_block, head_blocks;
};

// tokens_per_block tokens and heads_per_block heads a block: the cosines and sines are made
// once a block, one pair a thread, and used for all its heads.  Bound by memory: 3001 tokens of
// 40 x 128: 12.2 us, 5.0 TB/s; 1024 of 20 x 64: 3.7 us, a launch's latency.
__device__ void rope_block(const RopeRun& a, const RopeArgs& r, int64_t block, float* cosv, float* sinv) {
    const int64_t t0 = block / a.head_blocks * a.tokens_per_block;
    const int h0 = (int)(block % a.head_blocks) * a.heads_per_block;
    const int nt = (int)(a.T - t0 < a.tokens_per_block ? a.T - t0 : a.tokens_per_block);
    const int nh = a.heads - h0 < a.heads_per_block ? a.heads - h0 : a.heads_per_block;
    if (r.pos) {
        for (int i = threadIdx.x; i < nt * r.pairs; i += ROPE_THREADS) {
            const int t = i / r.pairs;
            const float2 cs = rope_turn(r, t0 + t, i - t * r.pairs);
            cosv[i] = cs.x;
            sinv[i] = cs.y;
        }
        __syncthreads();
    }
    const int pieces = a.head_dim >> 4, per_token = nh * pieces;
    for (int i = threadIdx.x; i < nt * per_token; i += ROPE_THREADS) {
        const int t = i / per_token, rest = i - t * per_token, h = rest / pieces;
        const Piece p = piece_of(r, rest - h * pieces);
        const int64_t head = (int64_t)(h0 + h) * a.head_dim;
        const uint16_t* src = a.x + (t0 + t) * a.x_stride + head;
        float lo[8], hi[8];
        widen8(*reinterpret_cast<const uint4*>(src + p.lo), lo);
        widen8(*reinterpret_cast<const uint4*>(src + p.hi), hi);
        if (p.pair >= 0 && r.pos) {
            const int at = t * r.pairs + p.pair;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                turn_in_piece(lo, hi, j, r.interleaved != 0, make_float2(cosv[at + j], sinv[at + j]));
        }
        uint16_t* dst = a.out + (t0 + t) * a.out_stride + head;
        *reinterpret_cast<uint4*>(dst + p.lo) = narrow8(lo);
        *reinterpret_cast<uint4*>(dst + p.hi) = narrow8(hi);
    }
}

__global__ __launch_bounds__(ROPE_THREADS) void rope_kernel(RopeRun a, RopeArgs r) {
    __shared__ float cosv[ROPE_LDS_PAIRS], sinv[ROPE_LDS_PAIRS];
    rope_block(a, r, blockIdx.x, cosv, sinv);
}

// ---------------------------------------------------------------- append

struct AppendArgs {
    w4a8_kv8 c;
    const int32_t* ctx_len;
    const int32_t* q_start;
    const uint16_t* k;
    const uint16_t* v;
    int64_t k_stride, v_stride, T, max_new;
    int64_t B;
    int pages_per_seq;        // pages that max_new tokens can touch
    int64_t cache_blocks;     // B * pages_per_seq * heads * 2
};

// The tokens of one page: positions first .. first + page_tokens - 1; the new ones are
// page places j0 .. j1 - 1 (from row `row` on), earlier ones 0 .. j0 - 1.
struct PageJob {
    int64_t page;      // -1: nothing to do
    int64_t row;
    int j0, j1;
};

__device__ __forceinline__ PageJob page_job(const AppendArgs& a, int64_t b, int w) {
    const int P = a.c.page_tokens;
    int64_t q0 = a.q_start[b], q1 = a.q_start[b + 1];
    q0 = q0 < 0 ? 0 : q0;
    q1 = q1 > a.T ? a.T : q1;
    if (q1 - q0 > a.max_new) q1 = q0 + a.max_new;
    const int64_t ctx = a.ctx_len[b];
    PageJob j{-1, 0, 0, 0};
    if (q1 <= q0 || ctx < 0) return j;
    const int64_t index = ctx / P + w, first = index * P, end = ctx + (q1 - q0);
    if (first >= end || index >= a.c.table_stride) return j;
    const int64_t page = a.c.table[b * a.c.table_stride + index];
    if (page < 0 || page >= a.c.pages) return j;
    j.page = page;
    j.j0 = (int)(ctx > first ? ctx - first : 0);
    j.j1 = (int)(end - first < P ? end - first : P);
    j.row = q0 + (first + j.j0 - ctx);
    return j;
}

// Block maximum of bit patterns of non-negative floats (NaN above inf above numbers).
__device__ __forceinline__ uint32_t block_top(uint32_t m, uint32_t* sm) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = m;
    __syncthreads();
    m = max(max(sm[0], sm[1]), max(sm[2], sm[3]));
    return m;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// rint(x / s) as IEEE quotient (by fp64 reciprocal, see div_by), in -127..127.
__device__ __forceinline__ int code_of(float x, double inv) {
    float q = __builtin_rintf(div_by(x, inv));
    return (int)__builtin_amdgcn_fmed3f(q, -127.0f, 127.0f);
}

__device__ __forceinline__ uint32_t pack4(const float* v, double inv) {
    return (uint32_t)(code_of(v[0], inv) & 0xFF) | (uint32_t)(code_of(v[1], inv) & 0xFF) << 8 |
           (uint32_t)(code_of(v[2], inv) & 0xFF) << 16 | (uint32_t)code_of(v[3], inv) << 24;
}

// Four stored codes brought from one scale to a larger one.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float c = (float)(int8_t)(w >> (8 * i)) * ratio;
        out |= (uint32_t)((int)__builtin_rintf(c) & 0xFF) << (8 * i);
    }
    return out;
}

// The new scale of a page, and what its codes are made with.
struct PageScale {
    float now, ratio;      // ratio: old codes to new ones (0 in a poisoned page)
    double inv;            // 0 where every code is 0
    bool grew;
};
__device__ __forceinline__ PageScale page_scale(uint32_t top, const float* stored, bool has_earlier) {
    const float old = has_earlier ? *stored : 0.0f;
    PageScale s;
    const float mine = __uint_as_float(top) / 127.0f;      // inf or NaN if any new value is
    const bool poisoned = !(mine <= 3.402823466e38f) || !(old <= 3.402823466e38f);
    s.now = poisoned ? __builtin_nanf("") : __builtin_fmaxf(mine, old);
    s.inv = poisoned || !(s.now > 0.0f) ? 0.0 : 1.0 / (double)s.now;
    s.grew = has_earlier && !(s.now == old);
    s.ratio = s.inv > 0.0 ? old / s.now : 0.0f;
    return s;
}

// NI: pieces of 16 elements a thread, page_tokens * head_dim / (16 * 256 threads) of them at most.

// Keys: a thread's pieces stay in registers between the page's maximum and the codes.
template <int NI>
__device__ void append_keys(const AppendArgs& a, const RopeArgs& r, const PageJob& job, int head, uint32_t* sm) {
    const int D = a.c.head_dim, P = a.c.page_tokens, pieces = D >> 4;
    const int n = (job.j1 - job.j0) * pieces;
    float lo[NI][8], hi[NI][8];
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < NI; ++e) {
        const int i = threadIdx.x + e * ROPE_THREADS;
        if (i < n) {
            const int t = i / pieces;
            const Piece p = piece_of(r, i - t * pieces);
            const uint16_t* src = a.k + (job.row + t) * a.k_stride + (int64_t)head * D;
            widen8(*reinterpret_cast<const uint4*>(src + p.lo), lo[e]);
            widen8(*reinterpret_cast<const uint4*>(src + p.hi), hi[e]);
            if (p.pair >= 0 && r.pos) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    turn_in_piece(lo[e], hi[e], j, r.interleaved != 0, rope_turn(r, job.row + t, p.pair + j));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, max(abs_bits(lo[e][j]), abs_bits(hi[e][j])));
        }
    }
    const int64_t ph = job.page * a.c.heads + head;
    int8_t* const page = a.c.k + ph * P * D;
    top = block_top(top, sm);
    const PageScale s = page_scale(top, a.c.k_scale + ph, job.j0 > 0);
    __syncthreads();                       // every thread has read the old scale
    if (threadIdx.x == 0) a.c.k_scale[ph] = s.now;
#pragma unroll
    for (int e = 0; e < NI; ++e) {
        const int i = threadIdx.x + e * ROPE_THREADS;
        if (i < n) {
            const int t = i / pieces;
            const Piece p = piece_of(r, i - t * pieces);
            int8_t* dst = page + (job.j0 + t) * D;
            const uint2 cl = s.inv > 0.0 ? make_uint2(pack4(lo[e], s.inv), pack4(lo[e] + 4, s.inv)) : make_uint2(0, 0);
            const uint2 ch = s.inv > 0.0 ? make_uint2(pack4(hi[e], s.inv), pack4(hi[e] + 4, s.inv)) : make_uint2(0, 0);
            *reinterpret_cast<uint2*>(dst + p.lo) = cl;
            *reinterpret_cast<uint2*>(dst + p.hi) = ch;
        }
    }
    if (s.grew)
        for (int i = threadIdx.x; i < job.j0 * D / 16; i += ROPE_THREADS) {
            uint4* w = reinterpret_cast<uint4*>(page) + i;
            const uint4 c = *w;
            *w = make_uint4(rescale4(c.x, s.ratio), rescale4(c.y, s.ratio), rescale4(c.z, s.ratio), rescale4(c.w, s.ratio));
        }
    if (job.j0 == 0)
        for (int i = threadIdx.x; i < (P - job.j1) * D / 16; i += ROPE_THREADS)
            reinterpret_cast<uint4*>(page + job.j1 * D)[i] = make_uint4(0, 0, 0, 0);
}

constexpr int VT_STRIDE = 128 + 16;        // bytes of a value row (tokens) in LDS

// Values: the codes go through LDS into token order, so a page row is written 16 tokens at
// a time.
template <int NI>
__device__ void append_values(const AppendArgs& a, const PageJob& job, int head, uint32_t* sm, uint8_t* vt) {
    const int D = a.c.head_dim, P = a.c.page_tokens, pieces = D >> 4;
    const int n = (job.j1 - job.j0) * pieces;
    float lo[NI][8], hi[NI][8];
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < NI; ++e) {
        const int i = threadIdx.x + e * ROPE_THREADS;
        if (i < n) {
            const int t = i / pieces, c = i - t * pieces;
            const uint16_t* src = a.v + (job.row + t) * a.v_stride + (int64_t)head * D + 16 * c;
            widen8(reinterpret_cast<const uint4*>(src)[0], lo[e]);
            widen8(reinterpret_cast<const uint4*>(src)[1], hi[e]);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, max(abs_bits(lo[e][j]), abs_bits(hi[e][j])));
        }
    }
    const int64_t ph = job.page * a.c.heads + head;
    int8_t* const page = a.c.v + ph * P * D;
    top = block_top(top, sm);
    const PageScale s = page_scale(top, a.c.v_scale + ph, job.j0 > 0);
#pragma unroll
    for (int e = 0; e < NI; ++e) {
        const int i = threadIdx.x + e * ROPE_THREADS;
        if (i < n) {
            const int t = i / pieces, c = i - t * pieces;
            uint8_t* dst = vt + (16 * c) * VT_STRIDE + job.j0 + t;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dst[j * VT_STRIDE] = s.inv > 0.0 ? (uint8_t)code_of(lo[e][j], s.inv) : 0;
                dst[(j + 8) * VT_STRIDE] = s.inv > 0.0 ? (uint8_t)code_of(hi[e][j], s.inv) : 0;
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) a.c.v_scale[ph] = s.now;
    const int chunks = P >> 4;
    for (int i = threadIdx.x; i < D * chunks; i += ROPE_THREADS) {
        const int d = i / chunks, c = i - d * chunks, j = 16 * c;      // places j .. j + 15 of row d
        if (j >= job.j1 && job.j0 > 0) continue;                       // past the end of a page that was begun earlier
        if (j + 16 <= job.j0 && !s.grew) continue;                     // earlier tokens, codes kept
        uint4* const dst = reinterpret_cast<uint4*>(page + d * P + j);
        const uint4 fresh = *reinterpret_cast<const uint4*>(vt + d * VT_STRIDE + j);
        uint4 old = make_uint4(0, 0, 0, 0);
        if (job.j0 > 0) old = *dst;
        uint32_t w[4] = {old.x, old.y, old.z, old.w};
        const uint32_t f[4] = {fresh.x, fresh.y, fresh.z, fresh.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int p = j + 4 * q;
            // bytes of the word that are new: places j0 .. j1 - 1
            uint32_t is_new = 0, is_old = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                is_new |= p + e >= job.j0 && p + e < job.j1 ? 0xFFu << (8 * e) : 0u;
                is_old |= p + e < job.j0 ? 0xFFu << (8 * e) : 0u;
            }
            uint32_t kept = w[q];
            if (s.grew) kept = (rescale4(kept, s.ratio) & is_old) | (kept & ~is_old);
            w[q] = (f[q] & is_new) | (kept & ~is_new);
        }
        *dst = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Blocks below cache_blocks each own one page of one sequence, one head, and its keys or its
// values, so nothing is shared between blocks (no atomics); the rest rotate the queries.
// 16 single tokens, 32 + 8 heads of 128: 5.6 us, the chain of dependent loads (lengths, page
// number, then, after the maximum, the old scale); 3265 tokens of three prompts: 21 us, 3.5 TB/s,
// where the queries alone take 11 and the pages alone 16 (512 threads a block changed nothing): by the
// counters vector issue takes 72 % of the time that a CU is busy and LDS 18 %, two thirds of it
// bank conflicts of the value codes' byte stores.
template <int NI>
__global__ __launch_bounds__(ROPE_THREADS) void kv8_append_kernel(AppendArgs a, RopeArgs r, RopeRun q) {
    __shared__ __attribute__((aligned(16))) uint8_t vt[128 * VT_STRIDE];
    __shared__ uint32_t sm[4];
    int64_t block = blockIdx.x;
    if (block >= a.cache_blocks) {
        float* const cosv = reinterpret_cast<float*>(vt);
        rope_block(q, r, block - a.cache_blocks, cosv, cosv + ROPE_LDS_PAIRS);
        return;
    }
    const int values = (int)(block & 1);
    block >>= 1;
    const int head = (int)(block % a.c.heads);
    block /= a.c.heads;
    const PageJob job = page_job(a, block / a.pages_per_seq, (int)(block % a.pages_per_seq));
    if (job.page < 0) return;
    if (values) append_values<NI>(a, job, head, sm, vt);
    else append_keys<NI>(a, r, job, head, sm);
}
static_assert(2 * ROPE_LDS_PAIRS * sizeof(float) <= 128 * VT_STRIDE, "cos and sin fit in the value buffer");

RopeArgs rope_args(const w4a8_rope* r, bool inverse) {
    RopeArgs a{};
    a.sign = inverse ? -1.0f : 1.0f;
    if (!r) return a;
    a.pos = r->pos;
    a.pos_stride = r->pos_stride;
    a.inv_freq = r->inv_freq;
    a.pairs = r->rotary_dim / 2;
    a.interleaved = r->interleaved;
    int end = 0;
    for (int i = 0; i < W4A8_ROPE_MAX_AXES; ++i) a.end[i] = end += i < r->axes ? r->sections[i] : 0;
    return a;
}

// Tokens a block so that every thread makes at most one cosine, heads split until a small
// batch gives two blocks a CU.
RopeRun rope_run(const void* x, void* out, int64_t T, int heads, int head_dim, int64_t x_stride, int64_t out_stride,
                 int pairs) {
    RopeRun a{};
    a.x = static_cast<const uint16_t*>(x);
    a.out = static_cast<uint16_t*>(out);
    a.T = T; a.x_stride = x_stride; a.out_stride = out_stride;
    a.heads = heads; a.head_dim = head_dim;
    static_assert(W4A8_ROPE_MAX_HEAD_DIM / 2 <= ROPE_LDS_PAIRS && 8 * 16 <= ROPE_LDS_PAIRS, "a block's cosines fit");
    a.tokens_per_block = std::max(1, std::min(8, ROPE_THREADS / std::max(pairs, 16)));
    const int64_t tb = (T + a.tokens_per_block - 1) / a.tokens_per_block;
    a.heads_per_block = heads;
    while (a.heads_per_block > 4 && tb * ((heads + a.heads_per_block - 1) / a.heads_per_block) < 512)
        a.heads_per_block = (a.heads_per_block + 1) / 2;
    a.head_blocks = (heads + a.heads_per_block - 1) / a.heads_per_block;
    return a;
}
int64_t rope_blocks(const RopeRun& a) {
    return (a.T + a.tokens_per_block - 1) / a.tokens_per_block * a.head_blocks;
}

}  // namespace

// Pages of one sequence that max_new tokens after any context can touch.
int64_t append_pages_per_seq(int64_t max_new, int page_tokens) {
    return max_new <= 0 ? 0 : (max_new + page_tokens - 2) / page_tokens + 1;
}

// Upper bound of the blocks of a launch (for the grid limit).
int64_t rope_grid(int64_t T, int heads, int head_dim, int pairs) {
    return rope_blocks(rope_run(nullptr, nullptr, T, heads, head_dim, 0, 0, pairs));
}

hipError_t launch_rope(const void* x, int64_t T, int heads, int head_dim, int64_t x_stride, const w4a8_rope* rope,
                       int inverse, void* out, int64_t out_stride, hipStream_t stream) {
    (void)hipGetLastError();   // clear a stale error so the check below is about this launch
    const RopeArgs r = rope_args(rope, inverse != 0);
    const RopeRun a = rope_run(x, out, T, heads, head_dim, x_stride, out_stride, r.pairs);
    hipLaunchKernelGGL(rope_kernel, dim3((unsigned)rope_blocks(a)), dim3(ROPE_THREADS), 0, stream, a, r);
    return hipGetLastError();
}

hipError_t launch_append(const w4a8_kv8& c, const int32_t* ctx_len, const int32_t* q_start, int64_t B, int64_t T,
                         int64_t max_new, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                         const void* q, int q_heads, int64_t q_stride, const w4a8_rope* rope, void* q_out,
                         int64_t out_stride, hipStream_t stream) {
    (void)hipGetLastError();
    const RopeArgs r = rope_args(rope, false);
    AppendArgs a{};
    a.c = c;
    a.ctx_len = ctx_len; a.q_start = q_start;
    a.k = static_cast<const uint16_t*>(k); a.v = static_cast<const uint16_t*>(v);
    a.k_stride = k_stride; a.v_stride = v_stride; a.T = T; a.max_new = max_new; a.B = B;
    a.pages_per_seq = (int)append_pages_per_seq(max_new, c.page_tokens);
    a.cache_blocks = B * a.pages_per_seq * c.heads * 2;
    RopeRun run{};
    int64_t blocks = a.cache_blocks;
    if (q) {
        run = rope_run(q, q_out, T, q_heads, c.head_dim, q_stride, out_stride, r.pairs);
        blocks += rope_blocks(run);
    }
    if (blocks == 0) return hipSuccess;
    const int pieces = c.page_tokens * c.head_dim / (16 * ROPE_THREADS);
    const dim3 grid((unsigned)blocks), threads(ROPE_THREADS);
    if (pieces <= 1) hipLaunchKernelGGL(kv8_append_kernel<1>, grid, threads, 0, stream, a, r, run);
    else if (pieces <= 2) hipLaunchKernelGGL(kv8_append_kernel<2>, grid, threads, 0, stream, a, r, run);
    else hipLaunchKernelGGL(kv8_append_kernel<4>, grid, threads, 0, stream, a, r, run);
    return hipGetLastError();
}

}  // namespace w4a8
