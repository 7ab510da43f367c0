// The gate between an expert's two products (gfx950): h = g sigmoid(g) u of
// the first product's halves (g, u), quantized 1x128 for the second product,
// with the 8-bit checkpoint of (g, u), and the backward pass from that
// checkpoint.
//
// sigmoid(g) = 1 / (1 + exp(-g));  with dh the gradient of h:
//   du = dh g sigmoid(g),   dg = dh u sigmoid(g) (1 + g (1 - sigmoid(g))).
#include "device_common.hpp"
#include "launch.hpp"

#include <math.h>

namespace fp8fg {

namespace gate_detail {

__device__ __forceinline__ float sigmoidf(float x) { return 1.0f / (1.0f + expf(-x)); }

template <int N>
__device__ __forceinline__ void load_once(const float* p, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const v4f a = ld_once<v4f>(p + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i + j] = a[j];
    }
}
template <int N>
__device__ __forceinline__ void load_once(const uint16_t* p, float (&v)[N]) {
    if constexpr (N == 4) {
        const u32x2_t a = ld_once<u32x2_t>(p);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            v[2 * j] = __uint_as_float(a[j] << 16);
            v[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const u32x4 a = ld_once<u32x4>(p + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i + 2 * j] = __uint_as_float(a[j] << 16);
                v[i + 2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
            }
        }
    }
}

// 16 values of a lane, eight lanes to a 128-group: the group's scale and the lane's codes
__device__ __forceinline__ u32x4 encode16(const float (&v)[16], float& sc) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
    sc = amax / 448.0f;
    const float rc = 1.0f / sc;
    u32x4 c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = encode4(v4f{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]}, sc, rc);
    return c;
}

// A workgroup takes 32 rows of one 128-channel group: eight lanes per row.
// Row r of buffer blockIdx.z exists when r < rows[blockIdx.z] (rows may be
// null: all of them).
template <class T>
__global__ __launch_bounds__(256) void swiglu(const T* __restrict__ gu, int64_t M, int64_t I,
                                              const int32_t* __restrict__ rows, uint8_t* __restrict__ q,
                                              float* __restrict__ s, uint8_t* __restrict__ qc, float* __restrict__ sc) {
    const int64_t b = blockIdx.z, kb = blockIdx.x, nb = I / kBlock;
    int64_t end = rows ? int64_t(rows[b]) : M;
    end = end < M ? end : M;
    const int64_t ch = kb * kBlock + (threadIdx.x & 7) * 16;
    for (int64_t m = int64_t(blockIdx.y) * 32 + (threadIdx.x >> 3); m < end; m += int64_t(gridDim.y) * 32) {
        const T* row = gu + (b * M + m) * 2 * I + ch;
        float g[16], u[16], h[16];
        load_once<16>(row, g);
        load_once<16>(row + I, u);
#pragma unroll
        for (int i = 0; i < 16; ++i) h[i] = g[i] * sigmoidf(g[i]) * u[i];
        float a;
        const u32x4 ch_code = encode16(h, a);
        st<u32x4>(q + (b * M + m) * I + ch, ch_code);
        if ((threadIdx.x & 7) == 0) s[(b * nb + kb) * M + m] = a;
        if (qc) {
            float sg, su;
            const u32x4 cg = encode16(g, sg), cu = encode16(u, su);
            uint8_t* c = qc + (b * M + m) * 2 * I + ch;
            st<u32x4>(c, cg);
            st<u32x4>(c + I, cu);
            if ((threadIdx.x & 7) == 0) {
                sc[(b * 2 * nb + kb) * M + m] = sg;
                sc[(b * 2 * nb + nb + kb) * M + m] = su;
            }
        }
    }
}

// The backward pass of a 128-row x 128-channel tile: the checkpoint decoded,
// dg, du and h formed once in registers, and quantized along the channels
// (dg, du: the next product's A operand) and along the rows, transposed (dg,
// du, h: the operands of the two weight gradients).  A thread holds eight
// rows of four channels; a row's 128 channels lie in 32 lanes, a channel's
// rows in 16 threads, whose maxima meet in LDS.  The transposed codes pass
// through LDS so that whole 128-byte row segments are written.
constexpr int kTileThreads = 512;

template <class T>
__global__ __launch_bounds__(kTileThreads) void swiglu_backward(
    const uint8_t* __restrict__ qc, const float* __restrict__ sc, const T* __restrict__ dh, int64_t M, int64_t I,
    const int32_t* __restrict__ rows, uint8_t* __restrict__ q, float* __restrict__ s, uint8_t* __restrict__ qt,
    float* __restrict__ st_, uint8_t* __restrict__ qh, float* __restrict__ sh) {
    __shared__ float part[3][16][kBlock];
    __shared__ float col[3][kBlock];
    __shared__ __align__(16) uint8_t codes[kBlock][kBlock + 16];
    const int t = threadIdx.x, c4 = (t & 31) * 4, r8 = (t >> 5) * 8;
    const int64_t nb = I / kBlock, kb = blockIdx.x, mb = blockIdx.y;
    int64_t end = rows ? int64_t(rows[0]) : M;
    end = end < M ? end : M;
    if (mb * kBlock >= end) return;
    const int64_t ch = kb * kBlock + c4;
    float d[3][8][4];              // dg, du, h
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t m = mb * kBlock + r8 + i;
        if (m < end) {
            const uint32_t wg = ld<uint32_t>(qc + m * 2 * I + ch), wu = ld<uint32_t>(qc + m * 2 * I + I + ch);
            const float fg = sc[kb * M + m], fu = sc[(nb + kb) * M + m];
            float e[4];
            load_once<4>(dh + m * I + ch, e);
            const v2f g01 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(wg, 1.0f, false);
            const v2f g23 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(wg, 1.0f, true);
            const v2f u01 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(wu, 1.0f, false);
            const v2f u23 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(wu, 1.0f, true);
            const float gg[4] = {g01[0] * fg, g01[1] * fg, g23[0] * fg, g23[1] * fg};
            const float uu[4] = {u01[0] * fu, u01[1] * fu, u23[0] * fu, u23[1] * fu};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float sg = sigmoidf(gg[j]);
                d[0][i][j] = e[j] * uu[j] * (sg * (1.0f + gg[j] * (1.0f - sg)));
                d[1][i][j] = e[j] * (gg[j] * sg);
                d[2][i][j] = gg[j] * sg * uu[j];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) d[k][i][j] = 0.0f;
        }
    }
    // along the channels
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t m = mb * kBlock + r8 + i;
            const v4f v = v4f{d[k][i][0], d[k][i][1], d[k][i][2], d[k][i][3]};
            const float a = halfwave_max(abs_max4(v)) / 448.0f;
            const uint32_t w = encode4(v, a, 1.0f / a);
            if (m < end) {
                st<uint32_t>(q + m * 2 * I + k * I + ch, w);
                if (c4 == 0) s[(k * nb + kb) * M + m] = a;
            }
        }
    // along the rows
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(d[k][i][j]));
            part[k][t >> 5][c4 + j] = a;
        }
    __syncthreads();
    if (t < 3 * kBlock) {
        const int k = t / kBlock, c = t % kBlock;
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) a = fmaxf(a, part[k][i][c]);
        a /= 448.0f;
        col[k][c] = a;
        if (k < 2)
            st_[mb * 2 * I + k * I + kb * kBlock + c] = a;
        else
            sh[mb * I + kb * kBlock + c] = a;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = col[k][c4 + j], r = 1.0f / a;
            u32x2_t w;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = encode4(v4f{d[k][4 * i][j], d[k][4 * i + 1][j], d[k][4 * i + 2][j], d[k][4 * i + 3][j]}, a, r);
            st<u32x2_t>(&codes[c4 + j][r8], w);
        }
        __syncthreads();
        uint8_t* out = k < 2 ? qt + (k * I + kb * kBlock) * M : qh + kb * kBlock * M;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int piece = t + kTileThreads * i;          // 128 channels x 8 pieces of 16 rows
            const int c = piece >> 3, off = (piece & 7) * 16;
            if (mb * kBlock + off < M)                        // M % 16 == 0: whole pieces
                st<u32x4>(out + c * M + mb * kBlock + off, ld<u32x4>(&codes[c][off]));
        }
    }
}

}  // namespace gate_detail

using namespace gate_detail;

hipError_t launch_swiglu(const void* gu, int bf16, int64_t G, int64_t M, int64_t I, const int32_t* rows, uint8_t* q,
                         float* s, uint8_t* qc, float* sc, hipStream_t stream) {
    int64_t groups = (M + 31) / 32;
    if (groups > 65535) groups = 65535;      // the kernel strides over the rest
    const dim3 grid(unsigned(I / kBlock), unsigned(groups), unsigned(G));
    if (bf16)
        return launch_kernel(swiglu<uint16_t>, grid, dim3(256), stream, static_cast<const uint16_t*>(gu), M, I, rows, q,
                             s, qc, sc);
    return launch_kernel(swiglu<float>, grid, dim3(256), stream, static_cast<const float*>(gu), M, I, rows, q, s, qc, sc);
}

hipError_t launch_swiglu_backward(const uint8_t* qc, const float* sc, const void* dh, int bf16, int64_t M, int64_t I,
                                  const int32_t* rows, uint8_t* q, float* s, uint8_t* qt, float* st, uint8_t* qh,
                                  float* sh, hipStream_t stream) {
    const dim3 grid(unsigned(I / kBlock), unsigned((M + kBlock - 1) / kBlock));
    if (bf16)
        return launch_kernel(swiglu_backward<uint16_t>, grid, dim3(kTileThreads), stream, qc, sc,
                             static_cast<const uint16_t*>(dh), M, I, rows, q, s, qt, st, qh, sh);
    return launch_kernel(swiglu_backward<float>, grid, dim3(kTileThreads), stream, qc, sc,
                         static_cast<const float*>(dh), M, I, rows, q, s, qt, st, qh, sh);
}

}  // namespace fp8fg
