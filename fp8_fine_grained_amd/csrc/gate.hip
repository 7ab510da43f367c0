// The gate between an expert's two products (gfx950): h = g sigmoid(g) u of
// the first product's halves (g, u), quantized 1x128 for the second product,
// with the 8-bit checkpoint of (g, u), and the backward pass from that
// checkpoint.
//
// sigmoid(g) = 1 / (1 + exp(-g));  with dh the gradient of h:
//   du = dh g sigmoid(g),   dg = dh u sigmoid(g) (1 + g (1 - sigmoid(g))).
#include "elementwise.hpp"
#include "launch.hpp"

namespace fp8fg {

namespace gate_detail {

// A workgroup takes 16 rows of one 128-channel group: 16 lanes per row, eight
// channels per lane (one 16-byte load of BF16).  Row r of buffer blockIdx.z exists when r <
// rows[blockIdx.z] (rows may be null: all of them).  Offsets within the 16
// rows fit 32 bits.  Bound by memory once the encoding is cheap: 66900 x 2048 with
// the checkpoint, 972 MB, 174 us, 5.6 TB/s (a plain copy 5.2); with an IEEE division and
// library exponential per element and per-element checks in the encoding it took 248 us.
// Few rows are bound by latency and a wave's instructions.  With 16 channels per
// lane (us, 16 / 8): FP32 with the checkpoint 351 / 258, FP32 without 308 / 211 (a lane's
// 64 bytes pass through the cache in four loads), BF16 182 / 181 and 130 / 122; masked,
// 32 x 128 rows of which 1 to 64 are used, 6.4 / 5.1.
constexpr int V = 8, kLanes = kBlock / V, kRows = 256 / kLanes;

template <class T, bool STREAM>
__global__ __launch_bounds__(256) void swiglu(const T* __restrict__ gu, int64_t M, int64_t I,
                                              const int32_t* __restrict__ rows, uint8_t* __restrict__ q,
                                              float* __restrict__ s, uint8_t* __restrict__ qc, float* __restrict__ sc) {
    typedef typename encoder_of<T>::type Enc;
    const int64_t b = blockIdx.z, kb = blockIdx.x, nb = I / kBlock;
    int64_t end = rows ? int64_t(rows[b]) : M;
    end = end < M ? end : M;
    const uint32_t r = threadIdx.x / kLanes, c = (threadIdx.x % kLanes) * V, in = r * uint32_t(I) + c;
    for (int64_t m0 = int64_t(blockIdx.y) * kRows; m0 < end; m0 += int64_t(gridDim.y) * kRows) {
        if (m0 + r >= end) return;
        const T* row = gu + (b * M + m0) * 2 * I + kb * kBlock;
        float g[V], u[V], h[V];
        load_n<V, true>(row + (in + r * uint32_t(I)), g);
        load_n<V, true>(row + I + (in + r * uint32_t(I)), u);
        // BF16: two values at a time.  Interleaved over all eight, as the compiler would, the
        // kernel is slower (us, with a checkpoint and without, in pairs / all): 170 / 179
        // and 113 / 128; FP32 the other way, 156 / 152
#pragma unroll
        for (int i = 0; i < V; ++i) {
            h[i] = gate_of(g[i], u[i]);
            if (sizeof(T) == 2 && (i & 1)) __builtin_amdgcn_sched_barrier(0);
        }
        float a;
        const auto codes = encode_lane<Derived>(h, a);
        st_out<STREAM>(q + (b * M + m0) * I + kb * kBlock + in, codes);
        if (c == 0) s[(b * nb + kb) * M + m0 + r] = a;
        if (qc) {
            float sg, su;
            const auto cg = encode_lane<Enc>(g, sg), cu = encode_lane<Enc>(u, su);
            uint8_t* out = qc + (b * M + m0) * 2 * I + kb * kBlock;
            st_out<STREAM>(out + (in + r * uint32_t(I)), cg);
            st_out<STREAM>(out + I + (in + r * uint32_t(I)), cu);
            if (c == 0) {
                sc[(b * 2 * nb + kb) * M + m0 + r] = sg;
                sc[(b * 2 * nb + nb + kb) * M + m0 + r] = su;
            }
        }
    }
}

// The backward pass of a 128-row x 128-channel tile: the checkpoint decoded,
// dg, du and h formed once in registers, and quantized along the channels
// (dg, du: the next product's A operand) and along the rows, transposed (dg,
// du, h: the operands of the two weight gradients).  A thread holds four rows
// of eight channels, so that a row's 128 channels are one 16-lane row (its
// maximum by DPP) and a channel's four rows one word of transposed codes.  A
// channel's maxima over a wave's 16 rows meet by swaps that reduce two values into one
// register each time, over the eight waves in LDS.  The transposed codes pass through
// LDS so that whole 128-byte row segments are written.  Everything is formed
// from one read of the checkpoint and dh: 67456 x 2048, 1.27 GB, 254 us, 5.0 TB/s.  The
// vector units are about as busy as the memory (about 50 instructions for each
// triple dg, du, h): the first form, with divisions and LDS shuffles, took 710 us.
constexpr int kTileThreads = 512;

// The transposed codes of a tile in LDS: word row4 of channel ch (rows 4 row4
// .. + 3), the 16-byte pieces of a channel swapped by channel run and odd and even
// channels by halves, so that a wave's stores (16 channel runs x 4 words) meet
// 64 different banks
__device__ __forceinline__ uint32_t code_word(uint32_t ch, uint32_t row4) {
    return (ch ^ ((ch >> 6) & 1)) * 32 + (((row4 >> 2) ^ ((ch >> 3) & 7)) << 2) + (row4 & 3);
}

template <class T>
struct GateRow {                   // a thread's eight channels of a row, as loaded
    u32x2_t g, u;
    u32x4 dh[sizeof(T) == 4 ? 2 : 1];
    float sg, su;
};
__device__ __forceinline__ float dh_of(const u32x4 (&w)[1], int j) {
    return __uint_as_float((j & 1) ? w[0][j >> 1] & 0xFFFF0000u : w[0][j >> 1] << 16);
}
__device__ __forceinline__ float dh_of(const u32x4 (&w)[2], int j) { return __uint_as_float(w[j >> 2][j & 3]); }

template <class T, bool STREAM>
__global__ __launch_bounds__(kTileThreads, 4) void swiglu_backward(
    const uint8_t* __restrict__ qc, const float* __restrict__ sc, const T* __restrict__ dh, int64_t M, int64_t I,
    const int32_t* __restrict__ rows, uint8_t* __restrict__ q, float* __restrict__ s, uint8_t* __restrict__ qt,
    float* __restrict__ st_, uint8_t* __restrict__ qh, float* __restrict__ sh) {
    __shared__ float part[8][3 * kBlock];
    __shared__ __align__(16) float gs[3 * kBlock], gr[3 * kBlock], grl[3 * kBlock];      // the channels' groups
    __shared__ __align__(16) uint32_t codes[3][kBlock * kBlock / 4];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const uint32_t c8 = (t & 15) * 8, r4 = (t >> 4) * 4;
    const int64_t nb = I / kBlock, kb = blockIdx.x, mb = blockIdx.y;
    int64_t end = rows ? int64_t(rows[0]) : M;
    end = end < M ? end : M;
    if (mb * kBlock >= end) return;
    const bool full = (mb + 1) * kBlock <= end;    // uniform: every row of the tile exists
    const int64_t m0 = mb * kBlock + r4;
    // offsets within the tile fit 32 bits (I <= 2^23)
    const uint8_t* qg = qc + mb * kBlock * 2 * I + kb * kBlock;
    const uint8_t* pd = reinterpret_cast<const uint8_t*>(dh + mb * kBlock * I + kb * kBlock);
    const float* sg_ = sc + kb * M + mb * kBlock;
    const float* su_ = sc + (nb + kb) * M + mb * kBlock;
    GateRow<T> in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // a row past the end: the tile's first row, with zeros in the place of its codes and dh
        const bool live = full || m0 + i < end;
        const uint32_t r = live ? r4 : 0u;
        const int64_t step = full ? i : 0;
        const uint32_t ri = full ? r : (live ? r + i : 0u);
        const uint32_t oc = ri * uint32_t(2 * I) + c8, od = (ri * uint32_t(I) + c8) * uint32_t(sizeof(T));
        in[i].g = ld_once<u32x2_t>(qg + step * 2 * I + oc);
        in[i].u = ld_once<u32x2_t>(qg + step * 2 * I + I + oc);
#pragma unroll
        for (int p = 0; p < int(sizeof(in[i].dh) / 16); ++p) in[i].dh[p] = ld_once<u32x4>(pd + step * I * sizeof(T) + od + 16 * p);
        in[i].sg = sg_[step + ri];
        in[i].su = su_[step + ri];
    }
    if (!full) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (m0 + i >= end) {
                in[i].g = in[i].u = u32x2_t{0u, 0u};
#pragma unroll
                for (int p = 0; p < int(sizeof(in[i].dh) / 16); ++p) in[i].dh[p] = u32x4{0u, 0u, 0u, 0u};
                in[i].sg = in[i].su = 0.0f;
            }
    }
    float d[3][4][8];              // dg, du, h
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const v2f g2 = (p & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(in[i].g[p >> 1], 1.0f, true)
                                   : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(in[i].g[p >> 1], 1.0f, false);
            const v2f u2 = (p & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(in[i].u[p >> 1], 1.0f, true)
                                   : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(in[i].u[p >> 1], 1.0f, false);
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const int j = 2 * p + o;
                const float g = g2[o] * in[i].sg, u = u2[o] * in[i].su, e = dh_of(in[i].dh, j);
                float rest;
                const float sg = sigmoid_fast(g, rest), si = g * sg;
                d[0][i][j] = e * __builtin_fmaf(si, rest, sg) * u;      // sg (1 + g (1 - sg)); e u alone might pass FP32's range
                d[1][i][j] = e * si;
                d[2][i][j] = si * u;
            }
        }
    }
    // the channels' maxima over the wave's rows
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        float a[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            a[j] = fmaxf(fmaxf(fabsf(d[k][0][j]), fabsf(d[k][1][j])), fmaxf(fabsf(d[k][2][j]), fabsf(d[k][3][j])));
        // halves: a[i] then holds channel 2 i on lanes 0..31 and 2 i + 1 on the others
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(a[2 * i]), __float_as_uint(a[2 * i + 1]), false, false);
            const uint32_t lo = w[0], hi = w[1];
            a[i] = fmaxf(__uint_as_float(lo), __uint_as_float(hi));
        }
        // 16-lane rows: a[i] holds what a[2 i] held on even rows and a[2 i + 1] on odd ones
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(a[2 * i]), __float_as_uint(a[2 * i + 1]), false, false);
            const uint32_t lo = w[0], hi = w[1];
            part[wave][k * kBlock + c8 + 2 * (2 * i + ((lane >> 4) & 1)) + (lane >> 5)] =
                fmaxf(__uint_as_float(lo), __uint_as_float(hi));
        }
        __builtin_amdgcn_sched_barrier(0);      // one of the three at a time: their registers would not fit
    }
    __syncthreads();
    if (t < 3 * kBlock) {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = fmaxf(a, part[i][t]);
        const Derived g(a);
        gs[t] = a = g.s;
        gr[t] = g.r;
        grl[t] = g.rl;
        if (t < 2 * kBlock)
            st_[mb * 2 * I + (t >> 7) * I + kb * kBlock + (t & 127)] = a;
        else
            sh[mb * I + kb * kBlock + (t & 127)] = a;
    }
    // along the channels
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint8_t* out = q + mb * kBlock * 2 * I + k * I + kb * kBlock;
        float a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) a[i] = fmaxf(a[i], fabsf(d[k][i][j]));
            const Derived g(lanes_max<16>(a[i]));
            a[i] = g.s;
            uint32_t w[2];
            g.encode<2>(d[k][i], w);
            if (full || m0 + i < end) st_out<STREAM>(out + i * 2 * I + (r4 * uint32_t(2 * I) + c8), u32x2_t{w[0], w[1]});
            __builtin_amdgcn_sched_barrier(0);
        }
        if (c8 == 0) {
            float* p = s + (k * nb + kb) * M + m0;
            if (m0 + 4 <= end) {
                st<v4f>(p, v4f{a[0], a[1], a[2], a[3]});
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (m0 + i < end) p[i] = a[i];
            }
        }
    }
    __syncthreads();
    // along the rows
    const uint32_t even = code_word(c8, r4 >> 2), odd = code_word(c8 + 1, r4 >> 2);    // channels c8 + 2 i are 64 words apart
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        float r[8], rl[8];
        load_n<8>(gr + k * kBlock + c8, r);
        load_n<8>(grl + k * kBlock + c8, rl);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x[4] = {d[k][0][j], d[k][1][j], d[k][2][j], d[k][3][j]};
            uint32_t w[1];
            Derived(gs[k * kBlock + c8 + j], r[j], rl[j]).encode<1>(x, w);
            codes[k][((j & 1) ? odd : even) + (j >> 1) * 64] = w[0];
            if (j & 1) __builtin_amdgcn_sched_barrier(0);
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        uint8_t* out = (k < 2 ? qt + (k * I + kb * kBlock) * M : qh + kb * kBlock * M) + mb * kBlock;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t piece = t + kTileThreads * i;          // 128 channels x 8 pieces of 16 rows
            const uint32_t c = piece >> 3, off = (piece & 7) * 16;
            if (full || mb * kBlock + off < M)                     // M % 16 == 0: whole pieces
                st_out<STREAM>(out + (c * uint32_t(M) + off), ld<u32x4>(&codes[k][code_word(c, off >> 2)]));
        }
    }
}

}  // namespace gate_detail

using namespace gate_detail;

hipError_t launch_swiglu(const void* gu, int bf16, int64_t G, int64_t M, int64_t I, const int32_t* rows, uint8_t* q,
                         float* s, uint8_t* qc, float* sc, hipStream_t stream) {
    int64_t groups = (M + kRows - 1) / kRows;
    if (groups > 65535) groups = 65535;      // the kernel strides over the rest
    const dim3 grid(unsigned(I / kBlock), unsigned(groups), unsigned(G));
    const bool stream_out = G * M * I * (qc ? 3 : 1) >= kStreamBytes;
#define FP8FG_GATE(T, S) \
    return launch_kernel(swiglu<T, S>, grid, dim3(256), stream, static_cast<const T*>(gu), M, I, rows, q, s, qc, sc)
    if (bf16) {
        if (stream_out) FP8FG_GATE(uint16_t, true);
        FP8FG_GATE(uint16_t, false);
    }
    if (stream_out) FP8FG_GATE(float, true);
    FP8FG_GATE(float, false);
#undef FP8FG_GATE
}

hipError_t launch_swiglu_backward(const uint8_t* qc, const float* sc, const void* dh, int bf16, int64_t M, int64_t I,
                                  const int32_t* rows, uint8_t* q, float* s, uint8_t* qt, float* st, uint8_t* qh,
                                  float* sh, hipStream_t stream) {
    const dim3 grid(unsigned(I / kBlock), unsigned((M + kBlock - 1) / kBlock));
    const bool stream_out = 5 * M * I >= kStreamBytes;
#define FP8FG_GATE(T, S)                                                                                              \
    return launch_kernel(swiglu_backward<T, S>, grid, dim3(kTileThreads), stream, qc, sc, static_cast<const T*>(dh), M, \
                         I, rows, q, s, qt, st, qh, sh)
    if (bf16) {
        if (stream_out) FP8FG_GATE(uint16_t, true);
        FP8FG_GATE(uint16_t, false);
    }
    if (stream_out) FP8FG_GATE(float, true);
    FP8FG_GATE(float, false);
#undef FP8FG_GATE
}

}  // namespace fp8fg
