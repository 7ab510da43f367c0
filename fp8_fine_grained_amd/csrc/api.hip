// C entry points of libfp8fg.so (declared in include/fp8fg.h).
//
// Every argument is checked on the host before anything is enqueued, in this
// order: NULL pointers, sizes and each call's multiple-of rules, 16-byte
// alignment, enum values.  A zero-sized problem returns FP8FG_OK without touching the
// HIP runtime, so these checks can be exercised on a machine without a GPU.
#include "fp8fg.h"
#include "launch.hpp"

#include <initializer_list>
#include <stdint.h>

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxElems = int64_t(1) << 40;
// K-blocks of the calls that always run the wide exact kernel, whose single
// FP32 accumulator keeps the 2^-14 S contract up to this many (gemm.hip)
constexpr int64_t kWideMaxKBlocks = 92;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// hipErrorInvalidConfiguration: a size whose grid is longer than a launch takes
inline int hip_status(hipError_t e) {
    return e == hipSuccess ? FP8FG_OK : e == hipErrorInvalidConfiguration ? FP8FG_ERR_UNSUPPORTED : FP8FG_ERR_HIP;
}

inline bool valid_out(int out_dtype) { return out_dtype == FP8FG_OUT_BF16 || out_dtype == FP8FG_OUT_FP32; }

}  // namespace

extern "C" {

int fp8fg_abi_version(void) { return FP8FG_ABI_VERSION; }

const char* fp8fg_status_string(int status) {
    switch (status) {
        case FP8FG_OK: return "ok";
        case FP8FG_ERR_NULL: return "null pointer argument";
        case FP8FG_ERR_SHAPE: return "invalid shape (negative size, or a size that breaks the call's multiple-of rule)";
        case FP8FG_ERR_ALIGN: return "pointer not 16-byte aligned";
        case FP8FG_ERR_UNSUPPORTED: return "unsupported argument value or size";
        case FP8FG_ERR_HIP: return "HIP runtime error at launch";
        default: return "unknown status";
    }
}

// the quantizers' checks, shared by the fp32 and bf16 entry points
static int quant_act(const void* x, int bf16, int64_t M, int64_t K, int transpose_out, uint8_t* q, float* s,
                     void* stream) {
    if (M > 0 && K > 0 && (!x || !q || !s)) return FP8FG_ERR_NULL;   // empty arrays may be NULL
    if (M < 0 || K < 0) return FP8FG_ERR_SHAPE;
    if (transpose_out != 0 && transpose_out != 1) return FP8FG_ERR_UNSUPPORTED;
    // the grouped axis: a multiple of 16 (a last partial group is allowed)
    if (transpose_out == 0 && K % 16 != 0) return FP8FG_ERR_SHAPE;
    if (transpose_out == 1 && M % 16 != 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(q) || !aligned16(s)) return FP8FG_ERR_ALIGN;
    if (M > kMaxDim || K > kMaxDim || (M > 0 && K > kMaxElems / M)) return FP8FG_ERR_UNSUPPORTED;
    if (transpose_out == 1 && ((K + 63) / 64 > 65535)) return FP8FG_ERR_UNSUPPORTED;
    if (M == 0 || K == 0) return FP8FG_OK;
    return hip_status(fp8fg::launch_quant_act(x, bf16, M, K, transpose_out, q, s, static_cast<hipStream_t>(stream)));
}

static int quant_weight(const void* w, int bf16, int64_t N, int64_t K, int transpose_out, uint8_t* q, float* s,
                        void* stream) {
    if (N > 0 && K > 0 && (!w || !q || !s)) return FP8FG_ERR_NULL;   // empty arrays may be NULL
    if (N < 0 || K < 0 || N % 16 != 0 || K % 16 != 0) return FP8FG_ERR_SHAPE;
    if (transpose_out != 0 && transpose_out != 1) return FP8FG_ERR_UNSUPPORTED;
    if (!aligned16(w) || !aligned16(q) || !aligned16(s)) return FP8FG_ERR_ALIGN;
    if (N > kMaxDim || K > kMaxDim || (N > 0 && K > kMaxElems / N)) return FP8FG_ERR_UNSUPPORTED;
    if ((N + 127) / 128 > 65535) return FP8FG_ERR_UNSUPPORTED;
    if (N == 0 || K == 0) return FP8FG_OK;
    return hip_status(
        fp8fg::launch_quant_weight(w, bf16, N, K, transpose_out, q, s, static_cast<hipStream_t>(stream)));
}

int fp8_quant_act_1x128(const float* x, int64_t M, int64_t K, int transpose_out, uint8_t* q, float* s,
                        void* stream) {
    return quant_act(x, 0, M, K, transpose_out, q, s, stream);
}

int fp8_quant_act_1x128_bf16(const uint16_t* x, int64_t M, int64_t K, int transpose_out, uint8_t* q, float* s,
                             void* stream) {
    return quant_act(x, 1, M, K, transpose_out, q, s, stream);
}

int fp8_quant_weight_128x128(const float* w, int64_t N, int64_t K, int transpose_out, uint8_t* q, float* s,
                             void* stream) {
    return quant_weight(w, 0, N, K, transpose_out, q, s, stream);
}

int fp8_quant_weight_128x128_bf16(const uint16_t* w, int64_t N, int64_t K, int transpose_out, uint8_t* q, float* s,
                                  void* stream) {
    return quant_weight(w, 1, N, K, transpose_out, q, s, stream);
}

int fp8_quant_fprop_operands(const void* x, int x_bf16, int64_t M, const void* w, int w_bf16, int64_t N, int64_t K,
                             uint8_t* qa, float* sa, uint8_t* qb, float* sb, void* stream) {
    // an operand with no elements may come with NULL pointers (never touched)
    if (M > 0 && K > 0 && (!x || !qa || !sa)) return FP8FG_ERR_NULL;
    if (N > 0 && K > 0 && (!w || !qb || !sb)) return FP8FG_ERR_NULL;
    if (M < 0 || N < 0 || K < 0 || K % 16 != 0 || N % 16 != 0) return FP8FG_ERR_SHAPE;
    if ((x_bf16 != 0 && x_bf16 != 1) || (w_bf16 != 0 && w_bf16 != 1)) return FP8FG_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(w) || !aligned16(qa) || !aligned16(sa) || !aligned16(qb) || !aligned16(sb))
        return FP8FG_ERR_ALIGN;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim || (M > 0 && K > kMaxElems / M) || (N > 0 && K > kMaxElems / N))
        return FP8FG_ERR_UNSUPPORTED;
    // one 1-D grid: weight blocks plus rowwise workgroups (at most 65535 row groups)
    const int64_t kbs = (K + 127) / 128;
    if (kbs * ((N + 127) / 128) + ((kbs + 3) / 4) * 65535 > 0x7FFFFFFF) return FP8FG_ERR_UNSUPPORTED;
    if (K == 0 || (M == 0 && N == 0)) return FP8FG_OK;
    return hip_status(fp8fg::launch_quant_fprop(x, x_bf16, M, w, w_bf16, N, K, qa, sa, qb, sb,
                                                static_cast<hipStream_t>(stream)));
}

int fp8_requant_act_tokenwise(const uint8_t* q, const float* s, int64_t M, int64_t K, uint8_t* qt, float* st,
                              void* stream) {
    if (!q || !s || !qt || !st) return FP8FG_ERR_NULL;
    if (M < 0 || K < 0 || M % 16 != 0 || K % 16 != 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(s) || !aligned16(qt) || !aligned16(st)) return FP8FG_ERR_ALIGN;
    if (M > kMaxDim || K > kMaxDim || (M > 0 && K > kMaxElems / M)) return FP8FG_ERR_UNSUPPORTED;
    if (K / 64 > 65535 || M / 128 > 0x7FFFFFFF) return FP8FG_ERR_UNSUPPORTED;
    if (M == 0 || K == 0) return FP8FG_OK;
    return hip_status(fp8fg::launch_requant_act_tokens(q, s, M, K, qt, st, static_cast<hipStream_t>(stream)));
}

int fp8_quant_mx_1x32(const float* x, int64_t R, int64_t K, uint8_t* q, uint8_t* e, void* stream) {
    if (!x || !q || !e) return FP8FG_ERR_NULL;
    if (R < 0 || K < 0 || K % 32 != 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(q) || !aligned16(e)) return FP8FG_ERR_ALIGN;
    if (R > kMaxDim || K > kMaxDim || (R > 0 && K > kMaxElems / R)) return FP8FG_ERR_UNSUPPORTED;
    if (R == 0 || K == 0) return FP8FG_OK;
    return hip_status(fp8fg::launch_quant_mx(x, R, K, q, e, static_cast<hipStream_t>(stream)));
}

int fp8_quant_mx_1x32_transposed(const float* x, int64_t M, int64_t K, uint8_t* q, uint8_t* e, void* stream) {
    if (M > 0 && K > 0 && (!x || !q || !e)) return FP8FG_ERR_NULL;   // empty arrays may be NULL
    if (M < 0 || K < 0 || M % 32 != 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(q) || !aligned16(e)) return FP8FG_ERR_ALIGN;
    if (M > kMaxDim || K > kMaxDim || (M > 0 && K > kMaxElems / M)) return FP8FG_ERR_UNSUPPORTED;
    if ((K + 63) / 64 > 65535) return FP8FG_ERR_UNSUPPORTED;
    if (M == 0 || K == 0) return FP8FG_OK;
    return hip_status(fp8fg::launch_quant_mx_tokens(x, M, K, q, e, static_cast<hipStream_t>(stream)));
}

int fp8_gemm_mx(const uint8_t* a, const uint8_t* ea, const uint8_t* b, const uint8_t* eb, void* c, int out_dtype,
                int64_t M, int64_t N, int64_t K, void* stream) {
    if (!a || !ea || !b || !eb || !c) return FP8FG_ERR_NULL;
    if (M < 0 || N < 0 || K < 0 || M % 4 != 0 || N % 256 != 0 || K % 64 != 0) return FP8FG_ERR_SHAPE;
    if (K == 0 && M > 0 && N > 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(ea) || !aligned16(b) || !aligned16(eb) || !aligned16(c)) return FP8FG_ERR_ALIGN;
    if (!valid_out(out_dtype)) return FP8FG_ERR_UNSUPPORTED;
    if (M > kMaxDim || N > kMaxDim || K >= (int64_t(1) << 24)) return FP8FG_ERR_UNSUPPORTED;
    if ((K / 32) * M > int64_t(0xFFFFFF00) || (K / 32) * N > int64_t(0xFFFFFF00)) return FP8FG_ERR_UNSUPPORTED;
    if (((M + 255) / 256) * (N / 256) > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return FP8FG_OK;
    fp8fg::GemmArgs args{a, reinterpret_cast<const float*>(ea), b, reinterpret_cast<const float*>(eb), c,
                         nullptr, M, N, K, 1};
    return hip_status(fp8fg::launch_gemm_mx(out_dtype == FP8FG_OUT_FP32, fp8fg::GemmMode::Dense, args,
                                            static_cast<hipStream_t>(stream)));
}

int fp8_grouped_gemm_contiguous_mx(const uint8_t* a, const uint8_t* ea, const uint8_t* b, const uint8_t* eb,
                                   const int32_t* group_offsets, int64_t G, int64_t M_total, int64_t N, int64_t K,
                                   void* c, int out_dtype, void* stream) {
    if (!a || !ea || !b || !eb || !group_offsets || !c) return FP8FG_ERR_NULL;
    if (G < 0 || M_total < 0 || N < 0 || K < 0 || M_total % 128 != 0 || N % 256 != 0 || K % 64 != 0)
        return FP8FG_ERR_SHAPE;
    if (K == 0 && M_total > 0 && N > 0 && G > 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(ea) || !aligned16(b) || !aligned16(eb) || !aligned16(c) ||
        !aligned16(group_offsets))
        return FP8FG_ERR_ALIGN;
    if (!valid_out(out_dtype)) return FP8FG_ERR_UNSUPPORTED;
    if (M_total > kMaxDim || N > kMaxDim || K >= (int64_t(1) << 24) || G > kMaxDim - 1) return FP8FG_ERR_UNSUPPORTED;
    if ((K / 32) * M_total > int64_t(0xFFFFFF00) || (K / 32) * N > int64_t(0xFFFFFF00)) return FP8FG_ERR_UNSUPPORTED;
    if ((M_total / 256 + G) * (N / 256) > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    if (G == 0 || M_total == 0 || N == 0) return FP8FG_OK;
    fp8fg::GemmArgs args{a, reinterpret_cast<const float*>(ea), b, reinterpret_cast<const float*>(eb), c,
                         group_offsets, M_total, N, K, G};
    return hip_status(fp8fg::launch_gemm_mx(out_dtype == FP8FG_OUT_FP32, fp8fg::GemmMode::Contig, args,
                                            static_cast<hipStream_t>(stream)));
}

int fp8_grouped_gemm_masked_mx(const uint8_t* a, const uint8_t* ea, const uint8_t* b, const uint8_t* eb,
                               const int32_t* masked_m, int64_t G, int64_t M_max, int64_t N, int64_t K, void* c,
                               int out_dtype, void* stream) {
    if (!a || !ea || !b || !eb || !masked_m || !c) return FP8FG_ERR_NULL;
    if (G < 0 || M_max < 0 || N < 0 || K < 0 || M_max % 4 != 0 || N % 256 != 0 || K % 64 != 0)
        return FP8FG_ERR_SHAPE;
    if (K == 0 && M_max > 0 && N > 0 && G > 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(ea) || !aligned16(b) || !aligned16(eb) || !aligned16(c) || !aligned16(masked_m))
        return FP8FG_ERR_ALIGN;
    if (!valid_out(out_dtype)) return FP8FG_ERR_UNSUPPORTED;
    if (M_max > kMaxDim || N > kMaxDim || K >= (int64_t(1) << 24) || G > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    if ((K / 32) * M_max > int64_t(0xFFFFFF00) || (K / 32) * N > int64_t(0xFFFFFF00)) return FP8FG_ERR_UNSUPPORTED;
    const int64_t tiles_per_group = ((M_max + 255) / 256) * (N / 256);
    if (tiles_per_group > 0 && G > kMaxDim / tiles_per_group) return FP8FG_ERR_UNSUPPORTED;
    if (G == 0 || M_max == 0 || N == 0) return FP8FG_OK;
    fp8fg::GemmArgs args{a, reinterpret_cast<const float*>(ea), b, reinterpret_cast<const float*>(eb), c, masked_m,
                         M_max, N, K, G};
    return hip_status(fp8fg::launch_gemm_mx(out_dtype == FP8FG_OUT_FP32, fp8fg::GemmMode::Masked, args,
                                            static_cast<hipStream_t>(stream)));
}

// the dense call's checks; engine 0 = exact, 1 = FP8 MFMA
static int gemm_dense(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb, int bscale_kind, void* c,
                      int out_dtype, int64_t M, int64_t N, int64_t K, void* stream, int engine) {
    if (!a || !sa || !b || !sb || !c) return FP8FG_ERR_NULL;
    if (M < 0 || N < 0 || K < 0 || N % 16 != 0 || K % 16 != 0) return FP8FG_ERR_SHAPE;
    if (K == 0 && M > 0 && N > 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(sa) || !aligned16(b) || !aligned16(sb) || !aligned16(c)) return FP8FG_ERR_ALIGN;
    if (bscale_kind != FP8FG_BSCALE_128x128 && bscale_kind != FP8FG_BSCALE_1x128) return FP8FG_ERR_UNSUPPORTED;
    if (!valid_out(out_dtype)) return FP8FG_ERR_UNSUPPORTED;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    if (((M + 127) / 128) * ((N + 127) / 128) > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return FP8FG_OK;
    fp8fg::GemmArgs args{a, sa, b, sb, c, nullptr, M, N, K, 1};
    return hip_status(fp8fg::launch_gemm(engine, fp8fg::GemmMode::Dense, bscale_kind == FP8FG_BSCALE_1x128,
                                         out_dtype == FP8FG_OUT_FP32, args, static_cast<hipStream_t>(stream)));
}

int fp8_gemm_blockscaled(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb, int bscale_kind,
                         void* c, int out_dtype, int64_t M, int64_t N, int64_t K, void* stream) {
    return gemm_dense(a, sa, b, sb, bscale_kind, c, out_dtype, M, N, K, stream, 0);
}

int fp8_gemm_blockscaled_fp8mfma(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                                 int bscale_kind, void* c, int out_dtype, int64_t M, int64_t N, int64_t K,
                                 void* stream) {
    return gemm_dense(a, sa, b, sb, bscale_kind, c, out_dtype, M, N, K, stream, 1);
}

int fp8_gemm_blockscaled_fp8out(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb, uint8_t* q,
                                float* s, int64_t M, int64_t N, int64_t K, void* stream) {
    if (!a || !sa || !b || !sb || !q || !s) return FP8FG_ERR_NULL;
    if (M < 0 || N < 0 || K < 0 || N % 256 != 0 || K % 16 != 0) return FP8FG_ERR_SHAPE;
    if (K == 0 && M > 0 && N > 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(sa) || !aligned16(b) || !aligned16(sb) || !aligned16(q) || !aligned16(s))
        return FP8FG_ERR_ALIGN;
    if (M > kMaxDim || N > kMaxDim || (K + 127) / 128 > kWideMaxKBlocks) return FP8FG_ERR_UNSUPPORTED;
    if (((K + 127) / 128) * M * 4 > int64_t(0xFFFFFFFF)) return FP8FG_ERR_UNSUPPORTED;
    if (((M + 255) / 256) * (N / 256) > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return FP8FG_OK;
    fp8fg::GemmArgs args{a, sa, b, sb, q, nullptr, M, N, K, 1, s};
    return hip_status(fp8fg::launch_gemm(0, fp8fg::GemmMode::Dense, 0, 2, args, static_cast<hipStream_t>(stream)));
}

int fp8_grouped_gemm_contiguous(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                                const int32_t* group_offsets, int64_t G, int64_t M_total, int64_t N, int64_t K,
                                void* c, int out_dtype, void* stream) {
    if (!a || !sa || !b || !sb || !group_offsets || !c) return FP8FG_ERR_NULL;
    if (G < 0 || M_total < 0 || N < 0 || K < 0 || M_total % 128 != 0 || N % 16 != 0 || K % 16 != 0)
        return FP8FG_ERR_SHAPE;
    if (K == 0 && M_total > 0 && N > 0 && G > 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(sa) || !aligned16(b) || !aligned16(sb) || !aligned16(c) ||
        !aligned16(group_offsets))
        return FP8FG_ERR_ALIGN;
    if (!valid_out(out_dtype)) return FP8FG_ERR_UNSUPPORTED;
    if (M_total > kMaxDim || N > kMaxDim || K > kMaxDim || G > kMaxDim - 1) return FP8FG_ERR_UNSUPPORTED;
    if ((M_total / 128) * ((N + 127) / 128) > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    if (G == 0 || M_total == 0 || N == 0) return FP8FG_OK;
    fp8fg::GemmArgs args{a, sa, b, sb, c, group_offsets, M_total, N, K, G};
    return hip_status(fp8fg::launch_gemm(0, fp8fg::GemmMode::Contig, 0, out_dtype == FP8FG_OUT_FP32, args,
                                         static_cast<hipStream_t>(stream)));
}

int fp8_grouped_gemm_contiguous_fp8out(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                                       const int32_t* group_offsets, int64_t G, int64_t M_total, int64_t N,
                                       int64_t K, uint8_t* q, float* s, void* stream) {
    if (!a || !sa || !b || !sb || !group_offsets || !q || !s) return FP8FG_ERR_NULL;
    if (G < 0 || M_total < 0 || N < 0 || K < 0 || M_total % 128 != 0 || N % 256 != 0 || K % 16 != 0)
        return FP8FG_ERR_SHAPE;
    if (K == 0 && M_total > 0 && N > 0 && G > 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(sa) || !aligned16(b) || !aligned16(sb) || !aligned16(q) || !aligned16(s) ||
        !aligned16(group_offsets))
        return FP8FG_ERR_ALIGN;
    if (M_total > kMaxDim || N > kMaxDim || G > kMaxDim - 1 || (K + 127) / 128 > kWideMaxKBlocks)
        return FP8FG_ERR_UNSUPPORTED;
    if (((K + 127) / 128) * M_total * 4 > int64_t(0xFFFFFFFF)) return FP8FG_ERR_UNSUPPORTED;
    if ((M_total / 128) * ((N + 127) / 128) > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    if (G == 0 || M_total == 0 || N == 0) return FP8FG_OK;
    fp8fg::GemmArgs args{a, sa, b, sb, q, group_offsets, M_total, N, K, G, s};
    return hip_status(fp8fg::launch_gemm(0, fp8fg::GemmMode::Contig, 0, 2, args, static_cast<hipStream_t>(stream)));
}

int fp8_grouped_gemm_masked(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                            const int32_t* masked_m, int64_t G, int64_t M_max, int64_t N, int64_t K, void* c,
                            int out_dtype, void* stream) {
    if (!a || !sa || !b || !sb || !masked_m || !c) return FP8FG_ERR_NULL;
    if (G < 0 || M_max < 0 || N < 0 || K < 0 || N % 16 != 0 || K % 16 != 0) return FP8FG_ERR_SHAPE;
    if (K == 0 && M_max > 0 && N > 0 && G > 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(sa) || !aligned16(b) || !aligned16(sb) || !aligned16(c) || !aligned16(masked_m))
        return FP8FG_ERR_ALIGN;
    if (!valid_out(out_dtype)) return FP8FG_ERR_UNSUPPORTED;
    if (M_max > kMaxDim || N > kMaxDim || K > kMaxDim || G > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    const int64_t tiles_per_group = ((M_max + 127) / 128) * ((N + 127) / 128);
    if (tiles_per_group > 0 && G > kMaxDim / tiles_per_group) return FP8FG_ERR_UNSUPPORTED;
    if (G == 0 || M_max == 0 || N == 0) return FP8FG_OK;
    fp8fg::GemmArgs args{a, sa, b, sb, c, masked_m, M_max, N, K, G};
    return hip_status(fp8fg::launch_gemm(0, fp8fg::GemmMode::Masked, 0, out_dtype == FP8FG_OUT_FP32, args,
                                         static_cast<hipStream_t>(stream)));
}

int fp8_tile_weights_decode(const uint8_t* q, int64_t G, int64_t N, int64_t K, uint8_t* q_tiled, void* stream) {
    if (G > 0 && N > 0 && K > 0 && (!q || !q_tiled)) return FP8FG_ERR_NULL;   // empty arrays may be NULL
    if (G < 0 || N < 0 || K < 0 || N % 256 != 0 || K % 64 != 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(q_tiled)) return FP8FG_ERR_ALIGN;
    if (G > kMaxDim || N > kMaxDim || K >= (int64_t(1) << 24)) return FP8FG_ERR_UNSUPPORTED;
    if (G == 0 || N == 0 || K == 0) return FP8FG_OK;
    if (G * N > kMaxElems / K) return FP8FG_ERR_UNSUPPORTED;
    return hip_status(fp8fg::launch_tile_weights_decode(q, G, N, K, q_tiled, static_cast<hipStream_t>(stream)));
}

int fp8_grouped_gemm_masked_tiled_mx(const uint8_t* a, const uint8_t* ea, const uint8_t* b_tiled, const uint8_t* eb,
                                     const int32_t* masked_m, int64_t G, int64_t M_max, int64_t N, int64_t K, void* c,
                                     int out_dtype, void* stream) {
    if (!a || !ea || !b_tiled || !eb || !masked_m || !c) return FP8FG_ERR_NULL;
    if (G < 0 || M_max < 0 || N < 0 || K < 0 || M_max % 4 != 0 || N % 256 != 0 || K % 64 != 0) return FP8FG_ERR_SHAPE;
    if (K == 0 && M_max > 0 && N > 0 && G > 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(ea) || !aligned16(b_tiled) || !aligned16(eb) || !aligned16(c) ||
        !aligned16(masked_m))
        return FP8FG_ERR_ALIGN;
    if (!valid_out(out_dtype)) return FP8FG_ERR_UNSUPPORTED;
    if (M_max > 128 || N > kMaxDim || K >= (int64_t(1) << 24) || G > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    if ((K / 32) * N > int64_t(0xFFFFFF00)) return FP8FG_ERR_UNSUPPORTED;
    if (N > 0 && G > kMaxDim / (2 * (N / 256))) return FP8FG_ERR_UNSUPPORTED;
    if (G * ((M_max + 63) / 64) > 4096) return FP8FG_ERR_UNSUPPORTED;
    if (G == 0 || M_max == 0 || N == 0) return FP8FG_OK;
    fp8fg::GemmArgs args{a, reinterpret_cast<const float*>(ea), b_tiled, reinterpret_cast<const float*>(eb), c,
                         masked_m, M_max, N, K, G};
    return hip_status(fp8fg::launch_gemm_masked_tiled(out_dtype == FP8FG_OUT_FP32, args,
                                                      static_cast<hipStream_t>(stream), true));
}

int fp8_grouped_gemm_masked_tiled_fp8out(const uint8_t* a, const float* sa, const uint8_t* b_tiled, const float* sb,
                                         const int32_t* masked_m, int64_t G, int64_t M_max, int64_t N, int64_t K,
                                         uint8_t* q, float* s, void* stream) {
    if (!a || !sa || !b_tiled || !sb || !masked_m || !q || !s) return FP8FG_ERR_NULL;
    if (G < 0 || M_max < 0 || N < 0 || K < 0 || N % 256 != 0 || K % 64 != 0) return FP8FG_ERR_SHAPE;
    if (K == 0 && M_max > 0 && N > 0 && G > 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(sa) || !aligned16(b_tiled) || !aligned16(sb) || !aligned16(q) || !aligned16(s) ||
        !aligned16(masked_m))
        return FP8FG_ERR_ALIGN;
    if (M_max > 128 || N > kMaxDim || (K + 127) / 128 > kWideMaxKBlocks || G > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    if (N > 0 && G > kMaxDim / (2 * (N / 256))) return FP8FG_ERR_UNSUPPORTED;
    if (G * ((M_max + 63) / 64) > 4096) return FP8FG_ERR_UNSUPPORTED;
    if (G == 0 || M_max == 0 || N == 0) return FP8FG_OK;
    fp8fg::GemmArgs args{a, sa, b_tiled, sb, q, masked_m, M_max, N, K, G, s};
    return hip_status(fp8fg::launch_gemm_masked_tiled(2, args, static_cast<hipStream_t>(stream)));
}

int fp8_grouped_gemm_masked_tiled(const uint8_t* a, const float* sa, const uint8_t* b_tiled, const float* sb,
                                  const int32_t* masked_m, int64_t G, int64_t M_max, int64_t N, int64_t K, void* c,
                                  int out_dtype, void* stream) {
    if (!a || !sa || !b_tiled || !sb || !masked_m || !c) return FP8FG_ERR_NULL;
    if (G < 0 || M_max < 0 || N < 0 || K < 0 || N % 256 != 0 || K % 64 != 0) return FP8FG_ERR_SHAPE;
    if (K == 0 && M_max > 0 && N > 0 && G > 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(sa) || !aligned16(b_tiled) || !aligned16(sb) || !aligned16(c) ||
        !aligned16(masked_m))
        return FP8FG_ERR_ALIGN;
    if (!valid_out(out_dtype)) return FP8FG_ERR_UNSUPPORTED;
    // the decode tile: buffers of at most 128 rows; 256 K bytes per n-tile stay below 4 GiB
    if (M_max > 128 || N > kMaxDim || (K + 127) / 128 > kWideMaxKBlocks || G > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    if (N > 0 && G > kMaxDim / (2 * (N / 256))) return FP8FG_ERR_UNSUPPORTED;
    // the decode kernel ranks at most 4096 (expert, 64-row m-tile) pairs
    if (G * ((M_max + 63) / 64) > 4096) return FP8FG_ERR_UNSUPPORTED;
    if (G == 0 || M_max == 0 || N == 0) return FP8FG_OK;
    fp8fg::GemmArgs args{a, sa, b_tiled, sb, c, masked_m, M_max, N, K, G};
    return hip_status(fp8fg::launch_gemm_masked_tiled(out_dtype == FP8FG_OUT_FP32, args,
                                                      static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------------------
// mixture-of-experts operators

constexpr int64_t kMaxTopk = 16, kMaxLocalExperts = 256, kMaxExperts = 1024;

static inline bool flag(int f) { return f == 0 || f == 1; }
static inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// the checks that both routing calls share
static int route_args(int64_t ld, int64_t T, int64_t E, int64_t topk, int logits_bf16, int score, int renormalize) {
    if (T < 0 || E < 1 || topk < 1 || topk > E || ld < E) return FP8FG_ERR_SHAPE;
    if (!flag(logits_bf16) || !flag(renormalize) || (score != FP8FG_SCORE_SOFTMAX && score != FP8FG_SCORE_SIGMOID))
        return FP8FG_ERR_UNSUPPORTED;
    if (E > kMaxExperts || topk > kMaxTopk || T > kMaxDim || ld > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    return FP8FG_OK;
}

int moe_route(const void* logits, int logits_bf16, int64_t ld, const float* bias, int64_t T, int64_t E, int64_t topk,
              int64_t n_groups, int64_t topk_groups, int group_top, int score, int renormalize, float scale,
              int32_t* idx, float* w, void* stream) {
    if (T > 0 && (!logits || !idx || !w)) return FP8FG_ERR_NULL;
    if (const int e = route_args(ld, T, E, topk, logits_bf16, score, renormalize)) return e;
    if (n_groups < 1 || topk_groups < 1 || topk_groups > n_groups || E % n_groups != 0 ||
        topk > topk_groups * (E / n_groups))
        return FP8FG_ERR_SHAPE;
    if (!aligned16(logits) || !aligned16(bias) || !aligned16(idx) || !aligned16(w)) return FP8FG_ERR_ALIGN;
    if (group_top != 1 && group_top != 2) return FP8FG_ERR_UNSUPPORTED;
    int64_t pow2 = 1;
    while (pow2 < n_groups && pow2 < 32) pow2 *= 2;
    if (pow2 > 16 || (E / n_groups) * pow2 > kMaxExperts) return FP8FG_ERR_UNSUPPORTED;
    if (T == 0) return FP8FG_OK;
    const fp8fg::RouteCall c{logits, logits_bf16, ld, T, E, topk, n_groups, topk_groups, group_top,
                             score == FP8FG_SCORE_SIGMOID, renormalize, scale, bias, idx, w};
    return hip_status(fp8fg::launch_route(c, static_cast<hipStream_t>(stream)));
}

int moe_route_backward(const void* logits, int logits_bf16, int64_t ld, const int32_t* idx, const float* dw, int64_t T,
                       int64_t E, int64_t topk, int score, int renormalize, float scale, void* dlogits, void* stream) {
    if (T > 0 && (!logits || !idx || !dw || !dlogits)) return FP8FG_ERR_NULL;
    if (const int e = route_args(ld, T, E, topk, logits_bf16, score, renormalize)) return e;
    if (!aligned16(logits) || !aligned16(idx) || !aligned16(dw) || !aligned16(dlogits)) return FP8FG_ERR_ALIGN;
    if (T == 0) return FP8FG_OK;
    const fp8fg::RouteCall c{logits, logits_bf16, ld, T, E, topk, 1, 1, 1, score == FP8FG_SCORE_SIGMOID, renormalize,
                             scale, nullptr, const_cast<int32_t*>(idx), nullptr};
    return hip_status(fp8fg::launch_route_backward(c, dw, dlogits, static_cast<hipStream_t>(stream)));
}

// sizes of [T][H] tokens with topk entries each, G local experts
static int rows_args(int64_t T, int64_t H, int64_t topk, int64_t G, int64_t R) {
    if (T < 0 || H < 0 || G < 0 || R < 0 || topk < 1) return FP8FG_ERR_SHAPE;
    if (topk > kMaxTopk || G > kMaxLocalExperts) return FP8FG_ERR_UNSUPPORTED;
    if (T > kMaxDim / topk || H > kMaxDim || R > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    if (H > 0 && (T > kMaxElems / H || R > kMaxElems / H)) return FP8FG_ERR_UNSUPPORTED;
    // waves are counted in 32 bits, one per token and 512 channels at the most (whether a launch takes them is
    // checked with its grid)
    if (T * ((H + 511) / 512) + 127 * G > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    return FP8FG_OK;
}

// the local experts' index range: any, as long as it can be formed
static inline bool first_ok(int64_t first) { return first >= 0 && first <= kMaxDim - kMaxLocalExperts; }

int fp8_moe_dispatch_contiguous(const void* x, int x_bf16, int64_t T, int64_t H, const int32_t* idx, int64_t topk,
                                int64_t first, int64_t G, int64_t M_total, uint8_t* q, float* s, int32_t* row_of,
                                int32_t* group_offsets, int32_t* counts, void* stream) {
    if (G > 0 && (!group_offsets || !counts)) return FP8FG_ERR_NULL;
    if (G > 0 && T > 0 && (!idx || !row_of || (H > 0 && (!x || !q || !s)))) return FP8FG_ERR_NULL;
    if (H % 16 != 0 || M_total % 128 != 0) return FP8FG_ERR_SHAPE;
    if (const int e = rows_args(T, H, topk, G, M_total)) return e;
    const int64_t n = T * topk;
    if (G > 0 && M_total < (n + 127 * (G < n ? G : n)) / 128 * 128) return FP8FG_ERR_SHAPE;
    if (!first_ok(first)) return FP8FG_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(idx) || !aligned16(q) || !aligned16(s) || !aligned16(row_of) ||
        !aligned16(group_offsets) || !aligned16(counts))
        return FP8FG_ERR_ALIGN;
    if (!flag(x_bf16)) return FP8FG_ERR_UNSUPPORTED;
    if (G == 0) return FP8FG_OK;
    return hip_status(fp8fg::launch_dispatch(x, x_bf16, T, H, idx, topk, first, G, M_total, 0, q, s, row_of,
                                             group_offsets, counts, static_cast<hipStream_t>(stream)));
}

int fp8_moe_dispatch_masked(const void* x, int x_bf16, int64_t T, int64_t H, const int32_t* idx, int64_t topk,
                            int64_t first, int64_t G, int64_t M_max, uint8_t* q, float* s, int32_t* row_of,
                            int32_t* masked_m, void* stream) {
    if (G > 0 && !masked_m) return FP8FG_ERR_NULL;
    if (G > 0 && T > 0 && (!idx || !row_of || (H > 0 && (!x || !q || !s)))) return FP8FG_ERR_NULL;
    if (H % 16 != 0 || M_max < 1) return FP8FG_ERR_SHAPE;
    if (G > 0 && M_max > kMaxDim / G) return FP8FG_ERR_UNSUPPORTED;
    if (const int e = rows_args(T, H, topk, G, G > 0 ? G * M_max : 0)) return e;
    if (!first_ok(first)) return FP8FG_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(idx) || !aligned16(q) || !aligned16(s) || !aligned16(row_of) || !aligned16(masked_m))
        return FP8FG_ERR_ALIGN;
    if (!flag(x_bf16)) return FP8FG_ERR_UNSUPPORTED;
    if (G == 0) return FP8FG_OK;
    return hip_status(fp8fg::launch_dispatch(x, x_bf16, T, H, idx, topk, first, G, G * M_max, M_max, q, s, row_of,
                                             nullptr, masked_m, static_cast<hipStream_t>(stream)));
}

int moe_combine(const void* y, int y_bf16, int64_t R, int64_t H, const int32_t* row_of, const float* w, int64_t T,
                int64_t topk, void* out, int out_dtype, void* stream) {
    if (T > 0 && H > 0 && (!row_of || !out || (R > 0 && !y))) return FP8FG_ERR_NULL;
    if (H % 8 != 0) return FP8FG_ERR_SHAPE;
    if (const int e = rows_args(T, H, topk, 0, R)) return e;
    if (!aligned16(y) || !aligned16(row_of) || !aligned16(w) || !aligned16(out)) return FP8FG_ERR_ALIGN;
    if (!flag(y_bf16) || !valid_out(out_dtype)) return FP8FG_ERR_UNSUPPORTED;
    if (T == 0 || H == 0) return FP8FG_OK;
    return hip_status(fp8fg::launch_combine(y, y_bf16, R, H, row_of, w, T, topk, out, out_dtype == FP8FG_OUT_FP32,
                                            static_cast<hipStream_t>(stream)));
}

int fp8_moe_combine_backward(const void* dout, int dout_bf16, int64_t T, int64_t H, const void* y, int y_bf16,
                             int64_t R, const int32_t* row_of, const float* w, int64_t topk,
                             const int32_t* group_offsets, const int32_t* counts, int64_t G, uint8_t* q, float* s,
                             float* dw, void* stream) {
    if (T > 0 && (!row_of || !w || !dw || (H > 0 && !dout))) return FP8FG_ERR_NULL;
    if (R > 0 && H > 0 && (!y || !q || !s)) return FP8FG_ERR_NULL;
    if (G > 0 && (!group_offsets || !counts)) return FP8FG_ERR_NULL;
    if (H % 16 != 0) return FP8FG_ERR_SHAPE;
    if (const int e = rows_args(T, H, topk, G, R)) return e;
    if (!aligned16(dout) || !aligned16(y) || !aligned16(row_of) || !aligned16(w) || !aligned16(group_offsets) ||
        !aligned16(counts) || !aligned16(q) || !aligned16(s) || !aligned16(dw))
        return FP8FG_ERR_ALIGN;
    if (!flag(dout_bf16) || !flag(y_bf16)) return FP8FG_ERR_UNSUPPORTED;
    if (T == 0 && (G == 0 || R == 0)) return FP8FG_OK;
    return hip_status(fp8fg::launch_combine_backward(dout, dout_bf16, T, H, y, y_bf16, R, row_of, w, topk, group_offsets,
                                                     counts, G, q, s, dw, static_cast<hipStream_t>(stream)));
}

int fp8_swiglu(const void* gu, int gu_bf16, int64_t G, int64_t M, int64_t I, const int32_t* rows, uint8_t* q, float* s,
               uint8_t* qc, float* sc, void* stream) {
    if (G > 0 && M > 0 && I > 0 && (!gu || !q || !s || !qc != !sc)) return FP8FG_ERR_NULL;
    if (G < 0 || M < 0 || I < 0 || I % 128 != 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(gu) || !aligned16(q) || !aligned16(s) || !aligned16(qc) || !aligned16(sc) || !aligned4(rows))
        return FP8FG_ERR_ALIGN;
    // the kernels' offsets within a tile fit 32 bits
    if (!flag(gu_bf16) || G > 65535 || M > kMaxDim || I > (int64_t(1) << 23)) return FP8FG_ERR_UNSUPPORTED;
    if (G == 0 || M == 0 || I == 0) return FP8FG_OK;
    if (M > kMaxElems / (2 * I) / G) return FP8FG_ERR_UNSUPPORTED;
    return hip_status(fp8fg::launch_swiglu(gu, gu_bf16, G, M, I, rows, q, s, qc, sc, static_cast<hipStream_t>(stream)));
}

int fp8_swiglu_backward(const uint8_t* qc, const float* sc, const void* dh, int dh_bf16, int64_t M, int64_t I,
                        const int32_t* rows, uint8_t* q, float* s, uint8_t* qt, float* st, uint8_t* qh, float* sh,
                        void* stream) {
    if (M > 0 && I > 0 && (!qc || !sc || !dh || !q || !s || !qt || !st || !qh || !sh)) return FP8FG_ERR_NULL;
    if (M < 0 || I < 0 || I % 128 != 0 || M % 16 != 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(qc) || !aligned16(sc) || !aligned16(dh) || !aligned16(q) || !aligned16(s) || !aligned16(qt) ||
        !aligned16(st) || !aligned16(qh) || !aligned16(sh) || !aligned4(rows))
        return FP8FG_ERR_ALIGN;
    if (!flag(dh_bf16) || M > int64_t(128) * 65535 || I > (int64_t(1) << 23)) return FP8FG_ERR_UNSUPPORTED;
    if (M == 0 || I == 0) return FP8FG_OK;
    if (M > kMaxElems / (2 * I)) return FP8FG_ERR_UNSUPPORTED;
    return hip_status(fp8fg::launch_swiglu_backward(qc, sc, dh, dh_bf16, M, I, rows, q, s, qt, st, qh, sh,
                                                    static_cast<hipStream_t>(stream)));
}

int fp8_grouped_gemm_wgrad(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                           const int32_t* group_offsets, int64_t G, int64_t M, int64_t N, int64_t R, float* c,
                           int accumulate, void* stream) {
    if (G > 0 && M > 0 && N > 0 && (!c || !group_offsets || (R > 0 && (!a || !sa || !b || !sb)))) return FP8FG_ERR_NULL;
    if (G < 0 || M < 0 || N < 0 || R < 0 || R % 128 != 0 || N % 16 != 0) return FP8FG_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(sa) || !aligned16(b) || !aligned16(sb) || !aligned16(c) || !aligned16(group_offsets))
        return FP8FG_ERR_ALIGN;
    if (!flag(accumulate) || M > kMaxDim || N > kMaxDim || R > kMaxDim || G > kMaxDim - 1) return FP8FG_ERR_UNSUPPORTED;
    if (G == 0 || M == 0 || N == 0) return FP8FG_OK;
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
    if (G > kMaxDim / tiles) return FP8FG_ERR_UNSUPPORTED;
    fp8fg::GemmArgs args{a, sa, b, sb, c, group_offsets, M, N, R, G, nullptr};
    args.accumulate = accumulate;
    return hip_status(fp8fg::launch_gemm(0, fp8fg::GemmMode::Wgrad, 1, 1, args, static_cast<hipStream_t>(stream)));
}

// ---- the key/value cache ----

// log2 of a page's tokens, -1 where they are no power of two in [16, 256]
static int page_log(int64_t page) {
    for (int l = 4; l <= 8; ++l)
        if (page == int64_t(1) << l) return l;
    return -1;
}

// n rows of `width` bytes, `step` bytes (at least width) apart
struct Span {
    const void* p;
    int64_t n, width, step;
};
static Span span(const void* p, int64_t bytes) { return {p, 1, bytes, bytes}; }
static Span ints(const void* p, int64_t n) { return span(p, 4 * n); }
// whether two of them share a byte: rows between one another's, as the heads of a fused projection, do not
static bool meet(Span a, Span b) {
    if (a.n <= 0 || b.n <= 0 || a.width <= 0 || b.width <= 0) return false;
    const int64_t d = int64_t(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));      // b's first row, from a's
    if (d >= (a.n - 1) * a.step + a.width || -d >= (b.n - 1) * b.step + b.width) return false;
    const auto up = [](int64_t x, int64_t y) { return x <= 0 ? -(-x / y) : (x + y - 1) / y; };
    if (a.step == b.step) {
        // row i of a and row i + k of b: k from the first on whose end lies behind a's start
        int64_t k = up(1 - b.width - d, a.step);
        if (k < 1 - a.n) k = 1 - a.n;
        return k < b.n && d + k * a.step < a.width;
    }
    if (a.n > b.n) return meet(b, a);
    for (int64_t i = 0; i < a.n; ++i) {
        const int64_t at = i * a.step - d;               // a's row, from b's first
        const int64_t j = at - b.width < 0 ? 0 : (at - b.width) / b.step + 1;
        if (j < b.n && j * b.step < at + a.width) return true;
    }
    return false;
}
// one of those that a call writes, on one that it reads (a workgroup would read what another has written) or
// on another that it writes
static bool overlap(std::initializer_list<Span> writes, std::initializer_list<Span> reads) {
    for (const Span* w = writes.begin(); w != writes.end(); ++w) {
        for (const Span& r : reads)
            if (meet(*w, r)) return true;
        for (const Span* other = writes.begin(); other != w; ++other)
            if (meet(*w, *other)) return true;
    }
    return false;
}

// B requests with a block table of `width` entries each
static int table_args(int64_t B, int64_t width, int64_t page) {
    if (B < 0 || width < 0) return FP8FG_ERR_SHAPE;
    // (positions are rounded up to whole tiles in 32 bits)
    if (page_log(page) < 0 || B > 65536 || (width > 0 && (B > kMaxDim / width || page > (kMaxDim - 255) / width))) return FP8FG_ERR_UNSUPPORTED;
    return FP8FG_OK;
}

int kv_assign_pages(const int32_t* have, const int32_t* add, int64_t B, const int32_t* free_pages, const int32_t* n_free,
                    int64_t F, int64_t page, int32_t* table, int64_t width, int64_t T, int32_t* lens, int32_t* cu,
                    int32_t* positions, int32_t* slots, int32_t* left, void* stream) {
    if (!n_free || !cu || !left || (F > 0 && !free_pages) || (T > 0 && (!positions || !slots))) return FP8FG_ERR_NULL;
    if (B > 0 && (!have || !add || !lens || (width > 0 && !table))) return FP8FG_ERR_NULL;
    if (F < 0 || T < 0) return FP8FG_ERR_SHAPE;
    if (const int e = table_args(B, width, page)) return e;
    if (!aligned16(have) || !aligned16(add) || !aligned16(free_pages) || !aligned4(n_free) || !aligned16(table) || !aligned16(lens) ||
        !aligned16(cu) || !aligned16(positions) || !aligned16(slots) || !aligned16(left))
        return FP8FG_ERR_ALIGN;
    if (F > kMaxDim || T >= int64_t(1) << 23) return FP8FG_ERR_UNSUPPORTED;
    if (overlap({ints(table, B * width), ints(lens, B), ints(cu, B + 1), ints(positions, T), ints(slots, T), ints(left, 2)},
                {ints(have, B), ints(add, B), ints(free_pages, F), ints(n_free, 1)}))
        return FP8FG_ERR_UNSUPPORTED;
    return hip_status(fp8fg::launch_kv_assign(have, add, B, free_pages, n_free, F, page_log(page), table, width, T, lens, cu, positions,
                                              slots, left, static_cast<hipStream_t>(stream)));
}

int kv_release_pages(const int32_t* done, const int32_t* lens, const int32_t* table, int64_t B, int64_t width, int64_t page,
                     int32_t* free_pages, int64_t F, const int32_t* n_free, int32_t* lens_out, int32_t* left, void* stream) {
    if (!n_free || !left || (F > 0 && !free_pages)) return FP8FG_ERR_NULL;
    if (B > 0 && (!done || !lens || !lens_out || (width > 0 && !table))) return FP8FG_ERR_NULL;
    if (F < 0) return FP8FG_ERR_SHAPE;
    if (const int e = table_args(B, width, page)) return e;
    if (!aligned16(done) || !aligned16(lens) || !aligned16(table) || !aligned16(free_pages) || !aligned4(n_free) || !aligned16(lens_out) ||
        !aligned16(left))
        return FP8FG_ERR_ALIGN;
    if (F > kMaxDim || overlap({ints(free_pages, F), ints(lens_out, B), ints(left, 1)},
                               {ints(done, B), ints(lens, B), ints(table, B * width), ints(n_free, 1)}))
        return FP8FG_ERR_UNSUPPORTED;
    return hip_status(fp8fg::launch_kv_release(done, lens, table, B, width, page_log(page), free_pages, F, n_free, lens_out, left,
                                               static_cast<hipStream_t>(stream)));
}

// [T][H][D] with rows ld elements of `size` bytes apart
static int rows_of_heads(int64_t T, int64_t H, int64_t D, int64_t ld, int size) {
    if (H > 0 && (ld < H * D || ld * size % 16 != 0)) return FP8FG_ERR_SHAPE;
    return ld > kMaxElems || (T > 0 && ld > kMaxElems / T) ? FP8FG_ERR_UNSUPPORTED : FP8FG_OK;
}

int rope(const void* q, int64_t ldq, void* q_out, int64_t ldqo, int64_t Hq, const void* k, int64_t ldk, void* k_out, int64_t ldko,
         int64_t Hkv, int x_bf16, const int32_t* positions, const float* freqs, int64_t T, int64_t D, int64_t rot, int interleaved,
         float scale, int inverse, void* stream) {
    if (T > 0 && ((Hq > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !k_out)) || !positions || !freqs)) return FP8FG_ERR_NULL;
    if (T < 0 || Hq < 0 || Hkv < 0 || D <= 0 || D % 8 != 0 || rot <= 0 || rot % 16 != 0 || rot > D) return FP8FG_ERR_SHAPE;
    if (!flag(x_bf16) || !flag(interleaved) || !flag(inverse) || rot > 256 || D > 1024 || Hq > 65535 || Hkv > 65535 || T > kMaxDim)
        return FP8FG_ERR_UNSUPPORTED;
    const int size = x_bf16 ? 2 : 4;
    for (const int e : {rows_of_heads(T, Hq, D, ldq, size), rows_of_heads(T, Hq, D, ldqo, size), rows_of_heads(T, Hkv, D, ldk, size),
                        rows_of_heads(T, Hkv, D, ldko, size)})
        if (e) return e;
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(k_out) || !aligned16(positions) || !aligned16(freqs))
        return FP8FG_ERR_ALIGN;
    if (T == 0 || Hq + Hkv == 0) return FP8FG_OK;
    // in place, or apart
    const auto heads = [&](const void* p, int64_t H, int64_t ld) { return Span{p, T, H * D * size, ld * size}; };
    const Span none = span(nullptr, 0), qi = heads(q, Hq, ldq), ki = heads(k, Hkv, ldk), qo = heads(q_out, Hq, ldqo), ko = heads(k_out, Hkv, ldko);
    if (meet(qo, q == q_out && ldq == ldqo ? none : qi) || meet(ko, k == k_out && ldk == ldko ? none : ki) || meet(qo, ki) || meet(ko, qi) ||
        overlap({qo, ko}, {ints(positions, T), span(freqs, 2 * rot)}))
        return FP8FG_ERR_UNSUPPORTED;
    return hip_status(fp8fg::launch_rope({q, k, q_out, k_out, ldq, ldk, ldqo, ldko, T, Hq, Hkv, D, rot, x_bf16, interleaved, inverse, scale,
                                          positions, freqs}, static_cast<hipStream_t>(stream)));
}

// the cache's own sizes
static int cache_args(int64_t n_pages, int64_t H, int64_t page, int64_t D) {
    if (n_pages < 0 || H < 0) return FP8FG_ERR_SHAPE;
    if (page_log(page) < 0 || (D != 64 && D != 128 && D != 192 && D != 256) || H > 65535) return FP8FG_ERR_UNSUPPORTED;
    return n_pages > kMaxDim / page || (n_pages > 0 && H > kMaxElems / (n_pages * page * D)) ? FP8FG_ERR_UNSUPPORTED : FP8FG_OK;
}

int fp8_kv_append(const void* k, int64_t ldk, const void* v, int64_t ldv, int x_bf16, const int32_t* slots, int64_t T, int64_t H,
                  int64_t D, int64_t page, int64_t n_pages, uint8_t* k_cache, float* k_scale, uint8_t* v_cache, float* v_scale,
                  void* stream) {
    if (T > 0 && H > 0 && (!k || !v || !slots || (n_pages > 0 && (!k_cache || !k_scale || !v_cache || !v_scale)))) return FP8FG_ERR_NULL;
    if (T < 0) return FP8FG_ERR_SHAPE;
    if (const int e = cache_args(n_pages, H, page, D)) return e;
    if (!flag(x_bf16) || T > kMaxDim) return FP8FG_ERR_UNSUPPORTED;
    for (const int e : {rows_of_heads(T, H, D, ldk, x_bf16 ? 2 : 4), rows_of_heads(T, H, D, ldv, x_bf16 ? 2 : 4)})
        if (e) return e;
    if (!aligned16(k) || !aligned16(v) || !aligned16(slots) || !aligned16(k_cache) || !aligned16(k_scale) || !aligned16(v_cache) ||
        !aligned16(v_scale))
        return FP8FG_ERR_ALIGN;
    if (T == 0 || H == 0 || n_pages == 0) return FP8FG_OK;
    const int64_t codes = n_pages * H * page * D, scales = 4 * n_pages * H, size = x_bf16 ? 2 : 4;
    if (overlap({span(k_cache, codes), span(k_scale, scales), span(v_cache, codes), span(v_scale, scales)},
                {Span{k, T, H * D * size, ldk * size}, Span{v, T, H * D * size, ldv * size}, ints(slots, T)}))
        return FP8FG_ERR_UNSUPPORTED;
    return hip_status(fp8fg::launch_kv_append({k, v, ldk, ldv, T, H, D, n_pages, x_bf16, page_log(page), slots, k_cache, v_cache, k_scale,
                                               v_scale}, static_cast<hipStream_t>(stream)));
}

// the sizes of an attention call, and what they are together
static int attend_args(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t page, int64_t width, fp8fg::AttendCall& c) {
    if (T < 0 || Hq < 0 || Hkv < 0 || (Hkv == 0 ? Hq != 0 : Hq % Hkv != 0)) return FP8FG_ERR_SHAPE;
    if (const int e = table_args(B, width, page)) return e;
    if (const int e = cache_args(0, Hkv, page, D)) return e;
    // query rows of a key/value head
    if (Hq > 65535 || T > kMaxDim || (Hkv > 0 && T * (Hq / Hkv) >= int64_t(1) << 24)) return FP8FG_ERR_UNSUPPORTED;
    c.T = T;
    c.B = B;
    c.Hq = Hq;
    c.Hkv = Hkv;
    c.D = D;
    c.page_log = page_log(page);
    c.width = width;
    return FP8FG_OK;
}

int fp8_kv_attention_workspace(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t page, int64_t width, int64_t* bytes) {
    if (!bytes) return FP8FG_ERR_NULL;
    fp8fg::AttendCall c{};
    if (const int e = attend_args(T, B, Hq, Hkv, D, page, width, c)) return e;
    *bytes = T == 0 || B == 0 || Hq == 0 ? 0 : fp8fg::attend_workspace(c);
    return FP8FG_OK;
}

int fp8_kv_attention(const uint16_t* q, int64_t ldq, const uint8_t* k_cache, const float* k_scale, const uint8_t* v_cache,
                     const float* v_scale, int64_t n_pages, int64_t page, const int32_t* table, int64_t width, const int32_t* cu,
                     const int32_t* lens, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, float scale, uint16_t* out,
                     float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
    const bool work = T > 0 && B > 0 && Hq > 0;
    if (work && (!q || !k_cache || !k_scale || !v_cache || !v_scale || !cu || !lens || !out || (width > 0 && !table))) return FP8FG_ERR_NULL;
    fp8fg::AttendCall c{};
    if (const int e = attend_args(T, B, Hq, Hkv, D, page, width, c)) return e;
    if (const int e = cache_args(n_pages, Hkv, page, D)) return e;
    if (work && n_pages == 0) return FP8FG_ERR_SHAPE;
    if (const int e = rows_of_heads(T, Hq, D, ldq, 2)) return e;
    if (!(scale >= 0.0f) || scale > 0x1p64f) return FP8FG_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(k_scale) || !aligned16(v_cache) || !aligned16(v_scale) || !aligned16(table) ||
        !aligned16(cu) || !aligned16(lens) || !aligned16(out) || !aligned16(lse) || !aligned16(workspace))
        return FP8FG_ERR_ALIGN;
    if (!work) return FP8FG_OK;
    const int64_t need = fp8fg::attend_workspace(c);
    if (need > 0 && !workspace) return FP8FG_ERR_NULL;
    if (workspace_bytes < need) return FP8FG_ERR_SHAPE;
    // (a row's queries are read by the workgroup that writes its output, or by an earlier launch: in place is sound)
    const int64_t codes = n_pages * Hkv * page * D, scales = 4 * n_pages * Hkv, row = 2 * Hq * D;
    const Span queries{q, T, row, 2 * ldq}, result = span(out, T * row), sums = span(lse, lse ? 4 * T * Hq : 0), scratch = span(workspace, need);
    if ((!(out == q && ldq == Hq * D) && meet(result, queries)) || meet(sums, queries) || meet(scratch, queries) ||
        overlap({result, sums, scratch}, {span(k_cache, codes), span(k_scale, scales), span(v_cache, codes), span(v_scale, scales),
                                          ints(table, B * width), ints(cu, B + 1), ints(lens, B)}))
        return FP8FG_ERR_UNSUPPORTED;
    c.q = q;
    c.ldq = ldq;
    c.kc = k_cache;
    c.ks = k_scale;
    c.vc = v_cache;
    c.vs = v_scale;
    c.table = table;
    c.cu = cu;
    c.lens = lens;
    c.n_pages = n_pages;
    c.scale = scale;
    c.out = out;
    c.lse = lse;
    c.workspace = workspace;
    return hip_status(fp8fg::launch_attend(c, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
