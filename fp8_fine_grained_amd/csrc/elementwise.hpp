// Device helpers of the operators around the grouped GEMMs (moe.hip, gate.hip):
// vector loads and stores, reductions over runs of lanes, the sigmoid and the
// quantizer's encoding of a thread's share of a group.
#pragma once

#include "device_common.hpp"

namespace fp8fg {

// N consecutive elements as fp32 (16-byte aligned; bf16 with N == 4: 8-byte);
// ONCE: with the non-temporal hint, for data read exactly once
template <int N, bool ONCE = false>
__device__ __forceinline__ void load_n(const float* p, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const v4f a = ONCE ? ld_once<v4f>(p + i) : ld<v4f>(p + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i + j] = a[j];
    }
}
template <int N, bool ONCE = false>
__device__ __forceinline__ void load_n(const uint16_t* p, float (&v)[N]) {
    if constexpr (N == 4) {
        const u32x2_t a = ONCE ? ld_once<u32x2_t>(p) : ld<u32x2_t>(p);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            v[2 * j] = __uint_as_float(a[j] << 16);
            v[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const u32x4 a = ONCE ? ld_once<u32x4>(p + i) : ld<u32x4>(p + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i + 2 * j] = __uint_as_float(a[j] << 16);
                v[i + 2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
            }
        }
    }
}
template <int N>
__device__ __forceinline__ void store_n(float* p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) st<v4f>(p + i, v4f{v[i], v[i + 1], v[i + 2], v[i + 3]});
}
template <int N>
__device__ __forceinline__ void store_n(uint16_t* p, const float (&v)[N]) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = bf16_bits(v[2 * i]) | (bf16_bits(v[2 * i + 1]) << 16);
    if constexpr (N == 4) {
        st<u32x2_t>(p, u32x2_t{w[0], w[1]});
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; i += 4) st<u32x4>(p + 2 * i, u32x4{w[i], w[i + 1], w[i + 2], w[i + 3]});
    }
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = uint16_t(bf16_bits(v)); }

// A value from another lane of the same 16-lane row, without LDS
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) { return __uint_as_float(dpp<CTRL>(__float_as_uint(v))); }
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;   // quad_perm, row_(half_)mirror

struct MaxOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};
struct SumOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// Reduction over runs of L lanes (1, 2, 4, 8, 16, 32 or 64), every lane gets
// the result.  Within a 16-lane row the partner comes by DPP: neighbour, next
// pair, then the mirror image of eight and of sixteen lanes, whose quads (halves)
// already agree.  Across rows the halves are swapped.
template <int L, class T, class Op>
__device__ __forceinline__ T lanes_reduce(T v, Op op) {
    if (L >= 2) v = op(v, dpp<kXor1>(v));
    if (L >= 4) v = op(v, dpp<kXor2>(v));
    if (L >= 8) v = op(v, dpp<kMirror8>(v));
    if (L >= 16) v = op(v, dpp<kMirror16>(v));
    if (L >= 32) {
        const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
        const uint32_t a = s[0], b = s[1];
        v = op(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
    }
    if (L >= 64) {
        const auto s = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
        const uint32_t a = s[0], b = s[1];
        v = op(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
    }
    return v;
}
template <int L, class T>
__device__ __forceinline__ T lanes_max(T v) { return lanes_reduce<L>(v, MaxOp()); }
template <int L>
__device__ __forceinline__ float lanes_sum(float v) { return lanes_reduce<L>(v, SumOp()); }

// 1 / (1 + exp(-x)), within about two roundings.  exp is 2^(-x log2 e) with the
// product's low part put back; the reciprocal's one Newton step takes the
// place of an IEEE division.  x is clamped where the result is 1 to FP32's last bit,
// or below FP32's smallest normal.
__device__ __forceinline__ float sigmoid_fast(float x) {
    constexpr float kHi = -0x1.715476p+0f, kLo = -0x1.4ae0c0p-26f, kLn2 = 0x1.62e430p-1f;      // -log2 e, ln 2
    x = __builtin_amdgcn_fmed3f(x, -88.0f, 100.0f);
    const float t = x * kHi;
    const float lo = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    const float d = 1.0f + __builtin_fmaf(e, lo * kLn2, e);
    const float r = __builtin_amdgcn_rcpf(d);
    return __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.0f), r);
}

// A quantization group: its scale s = RN32(amax / 448), and the ends lo, hi of
// a bracket of its reciprocal, r (1 -+ 2^-21) with r = RN32(1 / s).  Scales
// outside [2^-80, 2^80] get ends of opposite signs, which never agree; s == 0 (every
// element so small that its code is a signed zero) gets 0 and 0.
struct Group {
    float s, lo, hi;
};
// the power of two that brings a far scale back, 1 for the others
__device__ __forceinline__ float far_factor(float s) { return s < 0x1p-80f ? 0x1p64f : s > 0x1p80f ? 0x1p-64f : 1.0f; }
__device__ __forceinline__ Group make_group(float amax) {
    Group g;
    g.s = amax / 448.0f;
    const float k = far_factor(g.s), r = 1.0f / (g.s * k);
    g.lo = g.s == 0.0f ? 0.0f : r * (1.0f - 0x1p-21f);
    g.hi = g.s == 0.0f ? 0.0f : r * (k != 1.0f ? -1.0f : 1.0f + 0x1p-21f);
    return g;
}

// Codes of RN32(x / s) for 4 N elements of a group, bit for bit as encode4
// gives them.
//
// The quotient rounded to FP32 lies between x lo and x hi (each end is 2^-21 away,
// its own roundings and the quotient's together less than 2^-22), and rounding
// to E4M3 is monotone: where both ends have the same code it is the quotient's.
// That is two products and one conversion per element.  Otherwise (2^-16 of
// the elements) every quotient is formed: with r the rounded reciprocal of
// t = s k, one remainder step makes x r faithful and a second one correctly
// rounded (Markstein's theorem on division by a correctly rounded
// reciprocal; the remainders x k - y t are exact).  A zero's sign does not
// survive the remainder and is put back.
template <int N>
__device__ __forceinline__ void encode_run(const float (&x)[4 * N], const Group& g, uint32_t (&code)[N]) {
    uint32_t differ = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        code[i] = cvt4(x[4 * i] * g.lo, x[4 * i + 1] * g.lo, x[4 * i + 2] * g.lo, x[4 * i + 3] * g.lo);
        differ |= code[i] ^ cvt4(x[4 * i] * g.hi, x[4 * i + 1] * g.hi, x[4 * i + 2] * g.hi, x[4 * i + 3] * g.hi);
    }
    if (differ) {
        const float k = far_factor(g.s), t = g.s * k, r = 1.0f / t;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float xs = x[4 * i + j] * k;
                y[j] = xs * r;
                y[j] = __builtin_fmaf(__builtin_fmaf(-y[j], t, xs), r, y[j]);
                y[j] = __builtin_fmaf(__builtin_fmaf(-y[j], t, xs), r, y[j]);
                y[j] = copysignf(y[j], x[4 * i + j]);
            }
            code[i] = cvt4(y[0], y[1], y[2], y[3]);
        }
    }
}

// 16 consecutive values of a lane, eight lanes to a 128-group: the group's
// scale and the lane's codes
__device__ __forceinline__ u32x4 encode16(const float (&v)[16], float& sc) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
    const Group g = make_group(lanes_max<8>(amax));
    sc = g.s;
    uint32_t c[4];
    encode_run<4>(v, g, c);
    return u32x4{c[0], c[1], c[2], c[3]};
}

}  // namespace fp8fg
