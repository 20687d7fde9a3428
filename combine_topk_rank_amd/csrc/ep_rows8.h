// ep_rows8.h — device helpers of the operators that make bf16 values or 8-bit
// rows (EP_FMT_FP8_E4M3_B128) from floats: loads, roundings, block maxima.
#pragma once

#include "ep_common.h"

namespace ep {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kScaleBlock = 128;      // elements that share a scale
constexpr float kFp8Max = 448.0f;     // largest e4m3 value
constexpr float kAmaxMin = 1e-4f;     // least block maximum of a quantised row

__device__ inline float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ inline float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Two floats rounded to nearest even (v_cvt_pk_bf16_f32), lo in the low half.
__device__ inline uint32_t bf16_pack(float lo, float hi) {
    const bf16x2 p = __builtin_convertvector(f32x2{lo, hi}, bf16x2);
    return __builtin_bit_cast(uint32_t, p);
}

__device__ inline void unpack8(const u32x4 u, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(u[i]);
        f[2 * i + 1] = bf16_hi(u[i]);
    }
}

__device__ inline u32x4 pack8(const float* f) {
    return u32x4{bf16_pack(f[0], f[1]), bf16_pack(f[2], f[3]), bf16_pack(f[4], f[5]),
                 bf16_pack(f[6], f[7])};
}

// Codes of eight floats times inv, bytes in element order: round to nearest
// even, saturated (the conversion alone would make a product beyond +-448 a
// NaN).  A NaN product (of a NaN, or of an infinity in a block whose maximum is
// infinite) becomes 0x7F with the sign of its element; a lane without one, the
// rule, skips that step.
__device__ inline u32x2 fp8_pack8(const float* v, float inv) {
    int w[2] = {0, 0};
    float p[8], q[8];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        p[i] = v[i] * inv;
        nan |= p[i] != p[i];
        q[i] = __builtin_amdgcn_fmed3f(p[i], -kFp8Max, kFp8Max);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], w[i], false);
        w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], w[i], true);
    }
    if (nan) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (p[i] != p[i]) {
                const int sh = 8 * (i & 3);
                const uint32_t code = 0x7Fu | ((__float_as_uint(v[i]) >> 24) & 0x80u);
                w[i / 4] = (int)(((uint32_t)w[i / 4] & ~(0xFFu << sh)) | (code << sh));
            }
    }
    return u32x2{(uint32_t)w[0], (uint32_t)w[1]};
}

// Largest magnitude of eight floats; a NaN takes no part (fmaxf returns the
// other operand).
__device__ inline float amax8(const float* v) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}

// Reductions over aligned groups of N = 16 or 64 lanes, the result in every lane
// of the group: within 16 lanes by data-parallel moves (neighbours, pairs, then
// mirrored in 8 and in 16), across them by the row swaps of gfx950.
template <int CTRL>
__device__ inline uint32_t dpp_move(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}

template <int N, typename T, typename OP>
__device__ inline T group_reduce(T v, OP op) {
    static_assert((N == 16 || N == 64) && sizeof(T) == 4, "groups of 16 or 64 lanes");
    const auto step = [&](uint32_t other) { v = op(v, __builtin_bit_cast(T, other)); };
    step(dpp_move<0xB1>(__builtin_bit_cast(uint32_t, v)));    // quad_perm 1 0 3 2
    step(dpp_move<0x4E>(__builtin_bit_cast(uint32_t, v)));    // quad_perm 2 3 0 1
    step(dpp_move<0x141>(__builtin_bit_cast(uint32_t, v)));   // row_half_mirror
    step(dpp_move<0x140>(__builtin_bit_cast(uint32_t, v)));   // row_mirror
    if constexpr (N == 64) {
        uint32_t u = __builtin_bit_cast(uint32_t, v);
        u32x2 p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        v = op(__builtin_bit_cast(T, (uint32_t)p[0]), __builtin_bit_cast(T, (uint32_t)p[1]));
        u = __builtin_bit_cast(uint32_t, v);
        p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        v = op(__builtin_bit_cast(T, (uint32_t)p[0]), __builtin_bit_cast(T, (uint32_t)p[1]));
    }
    return v;
}

template <int N>
__device__ inline float group_max(float v) {
    return group_reduce<N>(v, [](float a, float b) { return fmaxf(a, b); });
}

template <int N>
__device__ inline float group_sum(float v) {
    return group_reduce<N>(v, [](float a, float b) { return a + b; });
}

template <int N>
__device__ inline int group_min(int v) {
    return group_reduce<N>(v, [](int a, int b) { return a < b ? a : b; });
}

}  // namespace ep
