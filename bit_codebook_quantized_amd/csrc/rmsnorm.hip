// rmsnorm_quant_act and rmsnorm_grad: the RMS norm in front of a W4A8 linear and its
// backward, fused with the residual addition and with the block rotation and int8
// quantisation of the activations (include/w4a8_block.h states the formulas).
//
// Layout: a block covers one row (K / 256 slots of 16 lanes, up to 1024 threads) or, for
// rows of at most 8 slots, several rows of a 16-slot block; a lane keeps its 16 columns in
// registers from the load to the store, so every input is read once.
#include <algorithm>
#include <type_traits>

#include "rmsnorm_device.hpp"

namespace w4a8 {
namespace {

// Slots of a block for rows of nb 256-column blocks, and the rows it covers.
__host__ __device__ constexpr int norm_rows(int nb) { return nb <= 16 ? 16 / nb : 1; }
__host__ __device__ constexpr int norm_slots(int nb) { return nb * norm_rows(nb); }

struct Place {   // of a lane's slot
    int row_local, blk;
};
__device__ __forceinline__ Place place_of(int slot, int nb) {
    const int r = slot / nb;
    return Place{r, slot - r * nb};
}

// Bound by memory: x and the residual are read once, h and the int8 rows written once (7 bytes an
// element with a bf16 stream), two barriers a row (sum of squares, maximum).  2048 x 4096 bf16:
// 14.1 us, 4.2 TB/s where a large copy reaches 4.9; 1237 x 12288 fp32: 42.4 us, 3.9 TB/s; one row
// of 4096: 3.8 us, which is latency.  2048 x 4096 without a residual 10.5 us (3 bytes an element, 2.4
// TB/s: the rotation and its barrier no longer hide), bf16 rows alone 8.6 us (3.9 TB/s), with a residual 13.8
// us (4.9 TB/s).  Occupancy hides the barriers: 7 blocks of a 4096-column row
// share a CU (20,992 bytes of LDS each).
// RES: the stream's type (uint16_t = bf16 bits, float), HAS_RES: whether there is a
// residual at all.
template <typename RES, bool HAS_RES>
__global__ __launch_bounds__(1024) void rmsnorm_quant_kernel(const uint16_t* __restrict__ x, const RES* residual,
                                                             const float* __restrict__ weight, int64_t M, int K,
                                                             float eps, float qmaxf, RES* h_out, float* rstd_out,
                                                             uint16_t* y_out, int8_t* __restrict__ xq,
                                                             float* __restrict__ xs) {
    extern __shared__ __attribute__((aligned(16))) float lds[];
    float* const ssum = lds;             // 64 slot sums
    float* const smax = lds + 64;        // 64 slot maxima
    float* const tile = lds + 128;       // NT_SLOT floats a slot

    const int tid = threadIdx.x, slot = tid >> 4, l16 = tid & 15;
    const int nb = K >> 8;
    const Place pl = place_of(slot, nb);
    const int64_t row = (int64_t)blockIdx.x * norm_rows(nb) + pl.row_local;
    const bool ok = row < M;
    const int col = pl.blk * 256 + l16 * 16;
    const int64_t at = row * K + col;
    float* const t = tile + slot * NT_SLOT;

    float v[16], w[16];
    load16(weight + col, w);
    if (ok) {
        load16(x + at, v);
        if constexpr (HAS_RES) {
            float r[16];
            load16(residual + at, r);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = r[i] + v[i];
            round16(v, residual);
            if (h_out) store16(h_out + at, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    }

    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = __builtin_fmaf(v[i], v[i], ss);
    ss = slot_sum(ss);
    if (l16 == 0) ssum[slot] = ss;
    __syncthreads();
    ss = slots_sum(ssum, pl.row_local * nb, nb);
    // a sum that is not finite poisons the row (rather than giving rstd = 0, a row of zeros)
    const float rstd = ss <= 3.402823466e38f ? 1.0f / __builtin_sqrtf(ss / (float)K + eps) : __builtin_nanf("");
    if (rstd_out && ok && pl.blk == 0 && l16 == 0) rstd_out[row] = rstd;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = v[i] * rstd * w[i];
    if (y_out && ok) store16(y_out + at, v);
    if (!xq) return;

    rotate_f32(v, l16, t);
    const float amax = slot_max(block_absmax(v, 0.0f));
    if (l16 == 0) smax[slot] = amax;
    __syncthreads();
    const float rmax = slots_top(smax, pl.row_local * nb, nb);
    const float scale = row_scale(rmax, qmaxf);
    const bool poisoned = row_poisoned(rmax);
    const double inv = poisoned ? 0.0 : 1.0 / (double)scale;
    if (ok && pl.blk == 0 && l16 == 0) xs[row] = scale;
    quant_store(v, inv, qmaxf, ok, poisoned, xq, row, K, pl.blk, l16, reinterpret_cast<uint8_t*>(t));
}

// One block takes rows blockIdx.x, + gridDim.x, ... (groups of norm_rows(nb) rows) and keeps
// the sum of its rows' dweight in registers; the partial rows, one a block, are added by the next
// kernel in a fixed order (no atomics: the same bits every time).
// Bound by memory: 14 bytes an element with an fp32 stream.  8192 x 4096 fp32: 95 us and 5 for
// dweight, 4.7 TB/s; 4096 x 4096 bf16: 35 us, 3.8 TB/s; 8192 x 512 bf16: 15 us; 2048 x 4096 bf16
// without grad_h 21.7 us, and without the rotation as well 20.9 us.  The weight's
// columns and the dweight sums hold 32 registers, so four waves share a SIMD.
template <typename RES, bool ROT, bool HAS_GH>
__global__ __launch_bounds__(1024) void rmsnorm_grad_kernel(const uint16_t* __restrict__ grad,
                                                            const RES* __restrict__ h,
                                                            const float* __restrict__ rstd,
                                                            const float* __restrict__ weight, const RES* grad_h,
                                                            int64_t M, int K, RES* dx, float* __restrict__ partial) {
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const int tid = threadIdx.x, slot = tid >> 4, l16 = tid & 15;
    const int nb = K >> 8, rows = norm_rows(nb);
    const Place pl = place_of(slot, nb);
    const int col = pl.blk * 256 + l16 * 16;
    float* const t = lds + 128 + slot * NT_SLOT;

    float w[16], dw[16];
    load16(weight + col, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[i] = 0.0f;

    const int64_t groups = (M + rows - 1) / rows;
    int turn = 0;
    for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x, turn ^= 1) {
        float* const sm = lds + 64 * turn;     // two in turn: one barrier a row is enough
        const int64_t row = grp * rows + pl.row_local;
        const bool ok = row < M;
        const int64_t at = row * K + col;
        float g[16], hv[16], gh[16];
        float r = 0.0f;
        if (ok) {
            load16(grad + at, g);
            load16(h + at, hv);
            if constexpr (HAS_GH) load16(grad_h + at, gh);
            r = rstd[row];
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) g[i] = hv[i] = gh[i] = 0.0f;
        }
        if constexpr (ROT) {
            rotate_f32(g, l16, t);
            slot_transpose(g, l16, t);
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            dw[i] = __builtin_fmaf(g[i], hv[i] * r, dw[i]);
            g[i] *= w[i];
            dot = __builtin_fmaf(g[i], hv[i], dot);
        }
        dot = slot_sum(dot);
        if (l16 == 0) sm[slot] = dot;
        __syncthreads();
        dot = slots_sum(sm, pl.row_local * nb, nb);
        const float c = r * r * (dot / (float)K);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float d = r * __builtin_fmaf(-hv[i], c, g[i]);
            g[i] = HAS_GH ? gh[i] + d : d;
        }
        if (ok) store16(dx + at, g);
    }
    if (!partial) return;
    if (rows > 1) {      // one partial row a block: its rows' sums are added in their order
        float* const all = lds + 128;
        __syncthreads();
        store16(all + pl.row_local * K + col, dw);
        __syncthreads();
        if (pl.row_local > 0) return;
        for (int r = 1; r < rows; ++r) {
            float other[16];
            load16(all + r * K + col, other);
#pragma unroll
            for (int i = 0; i < 16; ++i) dw[i] += other[i];
        }
    }
    store16(partial + (int64_t)blockIdx.x * K + col, dw);
}
static_assert(16 * 256 <= 16 * NT_SLOT, "the columns of 16 slots fit in their tiles");

// dweight[k] = sum over the partial rows: 64 columns a block, 4 a lane (256-byte row pieces), 64
// lanes down the rows, then their sums through LDS, each in a fixed order.
constexpr int DW_THREADS = 1024;
__global__ __launch_bounds__(DW_THREADS) void rmsnorm_dweight_kernel(const float* __restrict__ partial, int rows, int K,
                                                                     float* __restrict__ dweight) {
    __shared__ __attribute__((aligned(16))) float4 sm[64][16];
    const int c = threadIdx.x & 15, p = threadIdx.x >> 4;
    const float4* src = reinterpret_cast<const float4*>(partial + blockIdx.x * 64) + c;
    const int64_t stride = K / 4;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int r = p; r < rows; r += 64) {
        const float4 v = src[r * stride];
        a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
    }
    sm[p][c] = a;
#pragma unroll
    for (int half = 32; half > 0; half >>= 1) {
        __syncthreads();
        if (p < half) {
            const float4 v = sm[p + half][c];
            a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
            sm[p][c] = a;
        }
    }
    if (p == 0) reinterpret_cast<float4*>(dweight + blockIdx.x * 64)[c] = a;
}

size_t norm_lds(int nb) { return (128 + (size_t)norm_slots(nb) * NT_SLOT) * sizeof(float); }

// Blocks of the backward: as many as the chip holds at once (1024 threads a CU at these
// register counts), so each
// keeps its dweight sums over many rows.
int64_t grad_blocks(int64_t M, int nb) {
    const int64_t groups = (M + norm_rows(nb) - 1) / norm_rows(nb);
    const int64_t most = 256 * std::max(1, 1024 / (16 * norm_slots(nb)));
    return std::min(groups, most);
}

template <typename RES, bool HAS_RES>
hipError_t launch_norm(const void* x, const void* residual, const float* weight, int64_t M, int K, float eps, int qmax,
                       void* h, float* rstd, void* y, int8_t* xq, float* xs, hipStream_t stream) {
    const int nb = K >> 8;
    const int64_t grid = (M + norm_rows(nb) - 1) / norm_rows(nb);
    hipLaunchKernelGGL((rmsnorm_quant_kernel<RES, HAS_RES>), dim3((unsigned)grid), dim3(16 * norm_slots(nb)),
                       norm_lds(nb), stream, static_cast<const uint16_t*>(x), static_cast<const RES*>(residual),
                       weight, M, K, eps, (float)qmax, static_cast<RES*>(h), rstd, static_cast<uint16_t*>(y), xq, xs);
    return hipGetLastError();
}

template <typename RES, bool ROT, bool HAS_GH>
void launch_grad(const void* grad, const void* h, const float* rstd, const float* weight, const void* grad_h, int64_t M,
                 int K, void* dx, float* partial, int64_t grid, hipStream_t stream) {
    const int nb = K >> 8;
    hipLaunchKernelGGL((rmsnorm_grad_kernel<RES, ROT, HAS_GH>), dim3((unsigned)grid), dim3(16 * norm_slots(nb)),
                       norm_lds(nb), stream, static_cast<const uint16_t*>(grad), static_cast<const RES*>(h), rstd,
                       weight, static_cast<const RES*>(grad_h), M, K, static_cast<RES*>(dx), partial);
}

}  // namespace

// stream_f32: the residual stream's type.  M >= 1.
hipError_t launch_rmsnorm_quant(const void* x, const void* residual, int stream_f32, const float* weight, int64_t M,
                                int K, float eps, int qmax, void* h, float* rstd, void* y, int8_t* xq, float* xs,
                                hipStream_t stream) {
    (void)hipGetLastError();   // clear a stale error so the check below is about this launch
    if (!residual) return launch_norm<uint16_t, false>(x, residual, weight, M, K, eps, qmax, h, rstd, y, xq, xs, stream);
    if (stream_f32) return launch_norm<float, true>(x, residual, weight, M, K, eps, qmax, h, rstd, y, xq, xs, stream);
    return launch_norm<uint16_t, true>(x, residual, weight, M, K, eps, qmax, h, rstd, y, xq, xs, stream);
}

int64_t rmsnorm_grad_partial_rows(int64_t M, int K) { return grad_blocks(M, K >> 8); }

hipError_t launch_rmsnorm_grad(const void* grad, const void* h, int stream_f32, const float* rstd, const float* weight,
                               const void* grad_h, int64_t M, int K, int rot, void* dx, float* dweight,
                               float* partial, hipStream_t stream) {
    (void)hipGetLastError();
    const int64_t grid = grad_blocks(M, K >> 8);
    float* const part = dweight ? partial : nullptr;
    if (grid > 0) {
        auto go = [&](auto res, auto has_gh) {
            using RES = decltype(res);
            constexpr bool GH = decltype(has_gh)::value;
            if (rot) launch_grad<RES, true, GH>(grad, h, rstd, weight, grad_h, M, K, dx, part, grid, stream);
            else launch_grad<RES, false, GH>(grad, h, rstd, weight, grad_h, M, K, dx, part, grid, stream);
        };
        if (stream_f32) { if (grad_h) go(float{}, std::true_type{}); else go(float{}, std::false_type{}); }
        else { if (grad_h) go(uint16_t{}, std::true_type{}); else go(uint16_t{}, std::false_type{}); }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (dweight)
        hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3(K / 64), dim3(DW_THREADS), 0, stream, partial,
                           (int)rmsnorm_grad_partial_rows(M, K), K, dweight);
    return hipGetLastError();
}

}  // namespace w4a8
