// Device helpers of the RMS norm kernels: the block rotation in fp32, sums over a row, and
// the loads and stores of 16 consecutive columns.
//
// Layout: a slot is 16 lanes (one DPP row) and owns one 256-column block of a row.  Lane j
// holds columns 16j .. 16j + 15 ("by rows") for everything elementwise, so its accesses are
// 16 and 32 bytes wide; after the rotation it holds columns 16i + j, i = 0 .. 15
// ("by columns").  The 16 x 16 transpose between the two goes through the slot's own LDS,
// within one wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rotq_device.hpp"
#include "w4a8_device.hpp"

namespace w4a8 {

// A slot's 16 x 16 floats in LDS, rows padded to 20: 16-byte row writes and column reads
// of consecutive lanes then fall on different banks.
constexpr int NT_STRIDE = 20;
constexpr int NT_SLOT = 16 * NT_STRIDE;

// Radix-4 stage of H4 = J - 2R, halved: out_i = sum / 2 - a_(3 - i).  Four stages give the
// block product over 16.  Each output carries three fp32 roundings, so the block product is
// within about 12 * 2^-24 of the block's norm: the int8 step that follows is 2^-7 of the
// row's maximum.
__device__ __forceinline__ void radix4f(float& a0, float& a1, float& a2, float& a3) {
    const float s = (a0 + a1) + (a2 + a3);
    const float b0 = __builtin_fmaf(0.5f, s, -a3), b1 = __builtin_fmaf(0.5f, s, -a2);
    const float b2 = __builtin_fmaf(0.5f, s, -a1), b3 = __builtin_fmaf(0.5f, s, -a0);
    a0 = b0; a1 = b1; a2 = b2; a3 = b3;
}

__device__ __forceinline__ void radix16f(float (&v)[16]) {
#pragma unroll
    for (int g = 0; g < 4; ++g) radix4f(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
#pragma unroll
    for (int g = 0; g < 4; ++g) radix4f(v[g], v[g + 4], v[g + 8], v[g + 12]);
}

// t: the slot's NT_SLOT floats (16-byte aligned).  In: v by rows; out: v by columns, or the
// other way round (a transpose is its own inverse).
__device__ __forceinline__ void slot_transpose(float (&v)[16], int l16, float* t) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(t + l16 * NT_STRIDE + 4 * i) =
            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = t[i * NT_STRIDE + l16];
    wave_lds_sync();
}

// By rows in, by columns out.
__device__ __forceinline__ void rotate_f32(float (&v)[16], int l16, float* t) {
    radix16f(v);
    slot_transpose(v, l16, t);
    radix16f(v);
}

// Sum over a slot's 16 lanes, the same bits in every lane (each step adds a pair whose two
// sides hold the same two values).
__device__ __forceinline__ float slot_sum(float a) {
    a += __uint_as_float(row_dpp_u<0xB1>(__float_as_uint(a)));    // quad_perm [1, 0, 3, 2]
    a += __uint_as_float(row_dpp_u<0x4E>(__float_as_uint(a)));    // quad_perm [2, 3, 0, 1]
    a += __uint_as_float(row_dpp_u<0x141>(__float_as_uint(a)));   // row_half_mirror
    a += __uint_as_float(row_dpp_u<0x140>(__float_as_uint(a)));   // row_mirror
    return a;
}

// Sum of sm[s0 .. s0 + ns - 1] in a fixed order (sm 16-byte aligned).
__device__ __forceinline__ float slots_sum(const float* sm, int s0, int ns) {
    float a = 0.0f;
    if (((s0 | ns) & 3) == 0) {
        for (int s = s0; s < s0 + ns; s += 4) {
            const float4 v = *reinterpret_cast<const float4*>(sm + s);
            a += (v.x + v.y) + (v.z + v.w);
        }
    } else {
        for (int s = s0; s < s0 + ns; ++s) a += sm[s];
    }
    return a;
}

// Maximum of sm[s0 .. s0 + ns - 1], every entry >= +0 or +inf.
__device__ __forceinline__ float slots_top(const float* sm, int s0, int ns) {
    float a = 0.0f;
    if (((s0 | ns) & 3) == 0) {
        for (int s = s0; s < s0 + ns; s += 4) {
            const float4 v = *reinterpret_cast<const float4*>(sm + s);
            a = __builtin_fmaxf(a, __builtin_fmaxf(__builtin_fmaxf(v.x, v.y), __builtin_fmaxf(v.z, v.w)));
        }
    } else {
        for (int s = s0; s < s0 + ns; ++s) a = __builtin_fmaxf(a, sm[s]);
    }
    return a;
}

__device__ __forceinline__ void load16(const uint16_t* __restrict__ p, float (&v)[16]) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void load16(const float* __restrict__ p, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 a = reinterpret_cast<const float4*>(p)[i];
        v[4 * i] = a.x; v[4 * i + 1] = a.y; v[4 * i + 2] = a.z; v[4 * i + 3] = a.w;
    }
}

__device__ __forceinline__ void store16(uint16_t* p, const float (&v)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = f32x2_to_bf16x2(v[2 * i], v[2 * i + 1]);
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// v rounded to the type it will be stored in.
__device__ __forceinline__ void round16(float (&v)[16], const uint16_t*) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = f32x2_to_bf16x2(v[2 * i], v[2 * i + 1]);
        v[2 * i] = __uint_as_float(w << 16);
        v[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void round16(float (&)[16], const float*) {}

}  // namespace w4a8
