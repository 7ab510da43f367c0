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
// N consecutive elements as loaded, widened when they are used: a load under a
// branch then stays in flight past it
template <class T, int N>
struct Raw {
    static constexpr int W = N * int(sizeof(T)) / 16;
    u32x4 w[W];
    template <bool ONCE = false>
    __device__ __forceinline__ void load(const T* p) {
        const uint8_t* b = reinterpret_cast<const uint8_t*>(p);
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = ONCE ? ld_once<u32x4>(b + 16 * i) : ld<u32x4>(b + 16 * i);
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i >> 2][i & 3]);
        const uint32_t two = w[i >> 3][(i >> 1) & 3];
        return __uint_as_float((i & 1) ? two & 0xFFFF0000u : two << 16);
    }
};
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

// STREAM: stores with the non-temporal hint, for outputs that no L2 holds until
// they are read again
template <bool STREAM, typename V>
__device__ __forceinline__ void st_out(void* p, V v) {
    if constexpr (STREAM)
        __builtin_nontemporal_store(v, reinterpret_cast<V*>(p));
    else
        st<V>(p, v);
}
// Outputs of this many bytes stream: the eight L2s of 4 MB hold 32 MB together.
// Measured, us plain / streaming: the gate's backward 13.6 / 13.5 at 10 MB, 19.5 /
// 17.4 at 42 MB, 274 / 255 at 690 MB; dispatch 23.1 / 24.1 at 59 MB, 62.1 / 56.7
// at 172 MB; combine's backward 26.6 / 25.7 at 29 MB, 125.7 / 120.9 at 172 MB.
constexpr int64_t kStreamBytes = 32 << 20;

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

// exp(-x) as 2^(-x log2 e) with the product's low part put back.  x is clamped
// where 1 / (1 + exp(-x)) is 1 to FP32's last bit, or below FP32's smallest normal.
__device__ __forceinline__ float exp_minus(float x) {
    constexpr float kHi = -0x1.715476p+0f, kLo = -0x1.4ae0c0p-26f, kLn2 = 0x1.62e430p-1f;      // -log2 e, ln 2
    x = __builtin_amdgcn_fmed3f(x, -88.0f, 100.0f);
    const float t = x * kHi;
    const float lo = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(e, lo * kLn2, e);
}

// sigmoid(x) = 1 / (1 + exp(-x)), within about two roundings: the reciprocal's
// one Newton step takes the place of an IEEE division.  `rest` takes
// 1 - sigmoid(x) = exp(-x) sigmoid(x) with a small relative error of its own (the
// difference would lose it for large x).
__device__ __forceinline__ float sigmoid_fast(float x, float& rest) {
    const float e = exp_minus(x), d = 1.0f + e;
    const float r = __builtin_amdgcn_rcpf(d);
    const float sg = __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.0f), r);
    rest = e * sg;
    return sg;
}
__device__ __forceinline__ float sigmoid_fast(float x) {
    float rest;
    return sigmoid_fast(x, rest);
}

// g sigmoid(g) u: q = g / (1 + exp(-g)) and its remainder, with what the sum
// lost in rounding, both times u in one rounding, so that only the exponential's error
// and the last rounding remain (and no product passes FP32's range before the result does)
__device__ __forceinline__ float gate_of(float g, float u) {
    const float e = exp_minus(g), d = 1.0f + e;
    const float r = __builtin_amdgcn_rcpf(d), q = g * r;
    const float d_lost = e < 1.0f ? e - (d - 1.0f) : 1.0f - (d - e);
    const float rest = __builtin_fmaf(-q, d_lost, __builtin_fmaf(-q, d, g)) * r;
    return __builtin_fmaf(q, u, rest * u);
}

// cvt4 without clearing its result first: the conversion of a pair keeps the
// other half of its destination, which the second pair then overwrites
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, __builtin_bit_cast(int, a), false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

// RN32(a / 448) for results from 2^-80 on: the product with RN32(1 / 448)
// corrected once by its exact remainder.  a / 448 is never within 1/896 of a last
// place of the middle between two normal floats (448 = 7 * 64), far more than
// the corrected value's error.  (Subnormal results can be exact ties.)
__device__ __forceinline__ float scale_near(float a) {
    const float y = a * (1.0f / 448.0f);
    return __builtin_fmaf(__builtin_fmaf(-448.0f, y, a), 1.0f / 448.0f, y);
}

// Scales outside [2^-80, 2^80) (0 among them) and the power of two that brings
// a far one near: quotients by far scales are formed from scaled operands
__device__ __forceinline__ bool far_scale(float s) { return __float_as_uint(s) - 0x17800000u >= 0x50000000u; }
__device__ __forceinline__ float far_factor(float s) { return s < 1.0f ? 0x1p64f : 0x1p-64f; }

// E4M3 codes of RN32(x / s) for 4 N elements of a group, by exact quotients: with
// r the rounded reciprocal of s (of s k, and x k, for a far scale), one remainder step
// makes x r faithful and a second one correctly rounded (Markstein's theorem on
// division by a correctly rounded reciprocal; the remainders are exact).  A
// zero's sign does not survive the remainder and is put back.  A subnormal scale
// can be a third below amax / 448: the quotient saturates.
template <int N>
__device__ __forceinline__ void encode_exact(const float (&x)[4 * N], float s, uint32_t (&code)[N]) {
    const float k = far_scale(s) ? far_factor(s) : 1.0f, t = s * k, r = s == 0.0f ? 0.0f : 1.0f / t;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float xs = x[4 * i + j] * k;
            y[j] = xs * r;
            y[j] = __builtin_fmaf(__builtin_fmaf(-y[j], t, xs), r, y[j]);
            y[j] = __builtin_fmaf(__builtin_fmaf(-y[j], t, xs), r, y[j]);
            y[j] = copysignf(fminf(fabsf(y[j]), 448.0f), x[4 * i + j]);
        }
        code[i] = cvt4(y[0], y[1], y[2], y[3]);
    }
}

// The codes of a group's elements, bit for bit as encode4 gives them.  FP32
// elements: a bracket [lo, hi] = r (1 -+ 2^-21) of the reciprocal.  RN32(x / s)
// lies between x lo and x hi (the roundings of r, of the products and of the quotient
// are together less than 2^-22), and rounding to E4M3 is monotone: where both
// ends have the same code it is the quotient's.  That is two products
// and one conversion per element; the others (2^-16 of them, exact ties
// above all) take encode_exact.  Far scales get ends of opposite signs, which never
// agree.
struct Bracket {
    float s, lo, hi;
    __device__ __forceinline__ explicit Bracket(float amax) : s(scale_near(amax)) {
        const float r = __builtin_amdgcn_rcpf(s);
        lo = r * (1.0f - 0x1p-21f);
        hi = r * (1.0f + 0x1p-21f);
        if (far_scale(s)) {
            s = amax / 448.0f;
            lo = 1.0f;
            hi = -1.0f;
        }
    }
    template <int N>
    __device__ __forceinline__ void encode(const float (&x)[4 * N], uint32_t (&code)[N]) const {
        uint32_t differ = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            code[i] = codes4(x[4 * i] * lo, x[4 * i + 1] * lo, x[4 * i + 2] * lo, x[4 * i + 3] * lo);
            differ |= code[i] ^ codes4(x[4 * i] * hi, x[4 * i + 1] * hi, x[4 * i + 2] * hi, x[4 * i + 3] * hi);
        }
        if (differ) encode_exact<N>(x, s, code);
    }
};

// BF16 elements: exact ties between codes are common (ratios of 8-bit numbers:
// every seventh maximum makes one element in sixteen a tie), so a branch on them
// would be taken by most waves.  The quotient itself is formed instead, from the
// reciprocal in two parts r + rl, r below 1 / s so that a zero keeps its sign:
// x rl + x r, one rounding, is within 2^-40 of x / s before it.  That decides
// the code: x = X 2^i and s = RN32(A 2^j / 448) with 8-bit X and A put x / s at
// least 2^-32 away from the middle of a code boundary and its FP32 neighbour, where
// RN32 would turn (the low bits of A / 7 repeat 001, 010 or 100, or are zero).
struct Ratio {
    float s, r, rl;
    __device__ __forceinline__ explicit Ratio(float amax) : s(scale_near(amax)) {
        r = __builtin_amdgcn_rcpf(s);
        r = __builtin_fmaf(r, -0x1p-22f, r);
        rl = r * __builtin_fmaf(-s, r, 1.0f);
        if (far_scale(s)) s = amax / 448.0f;
    }
    template <int N>
    __device__ __forceinline__ void encode(const float (&x)[4 * N], uint32_t (&code)[N]) const {
        if (far_scale(s)) {
            encode_exact<N>(x, s, code);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = __builtin_fmaf(x[4 * i + j], r, x[4 * i + j] * rl);
                code[i] = codes4(y[0], y[1], y[2], y[3]);
            }
        }
    }
};

// Values formed in FP32 here (a gate, a gradient): the same two-part quotient,
// within half a last place and 2^-40 of x / s, which differs from RN32(x / s) far less
// than the value's own roundings do.  For a far scale r and rl are those of s k, rl
// with its sign set, and the operands are scaled; a subnormal scale can be a
// third below amax / 448, so there the quotient saturates.
struct Derived {
    float s, r, rl;
    __device__ __forceinline__ explicit Derived(float amax) : s(scale_near(amax)) {
        if (far_scale(s)) {
            s = amax / 448.0f;
            const float t = s * far_factor(s);
            r = s == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(t) * (1.0f - 0x1p-22f);
            rl = s == 0.0f ? 0.0f : -r * __builtin_fmaf(-t, r, 1.0f);
        } else {
            r = __builtin_amdgcn_rcpf(s);
            r = __builtin_fmaf(r, -0x1p-22f, r);
            rl = r * __builtin_fmaf(-s, r, 1.0f);
        }
    }
    __device__ __forceinline__ Derived(float s_, float r_, float rl_) : s(s_), r(r_), rl(rl_) {}
    template <int N>
    __device__ __forceinline__ void encode(const float (&x)[4 * N], uint32_t (&code)[N]) const {
        float y[4 * N];
        if (rl >= 0.0f) {
#pragma unroll
            for (int i = 0; i < 4 * N; ++i) y[i] = __builtin_fmaf(x[i], r, x[i] * rl);
        } else {
            const float k = far_factor(s);
#pragma unroll
            for (int i = 0; i < 4 * N; ++i) {
                const float xs = x[i] * k;
                y[i] = __builtin_amdgcn_fmed3f(__builtin_fmaf(xs, r, xs * -rl), -448.0f, 448.0f);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) code[i] = codes4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    }
};

// N = 8 or 4 consecutive values of a lane, 128 / N lanes to a group: the group's
// scale and the lane's codes (G: Bracket, Ratio for values that are BF16, or Derived)
typedef uint32_t u32x1_t __attribute__((ext_vector_type(1)));
template <int N>
struct code_words {
    typedef u32x2_t type;
};
template <>
struct code_words<4> {
    typedef u32x1_t type;
};
template <class G, int N>
__device__ __forceinline__ typename code_words<N>::type encode_lane(const float (&v)[N], float& sc) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) amax = fmaxf(amax, fabsf(v[i]));
    const G g(lanes_max<128 / N>(amax));
    sc = g.s;
    uint32_t c[N / 4];
    g.template encode<N / 4>(v, c);
    typename code_words<N>::type w;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = c[i];
    return w;
}
// the encoding of values read as T
template <class T>
struct encoder_of {
    typedef Bracket type;
};
template <>
struct encoder_of<uint16_t> {
    typedef Ratio type;
};

}  // namespace fp8fg
