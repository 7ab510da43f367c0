// The operators around the grouped GEMMs of a mixture-of-experts layer
// (gfx950): the router's choice of experts and its gradient, the tokens' rows
// quantized into the layouts the grouped GEMMs read, and the weighted sum that
// brings the rows back, with its backward pass.
#include "elementwise.hpp"
#include "launch.hpp"

#include <math.h>

namespace fp8fg {

namespace moe_detail {

// ---------------------------------------------------------------------------
// Routing.  s = sigmoid(x) or softmax(x) over the row, c = s + bias; a group
// of experts scores the sum of its group_top (1 or 2) largest c; the
// topk_groups best groups keep their experts, and the topk largest c among
// them are chosen, equal ones by the lowest index.  An expert with c = -inf
// (a logit of -inf) is never chosen; where fewer than topk remain the index
// is -1 and the weight 0.  Weights are scale * s, divided by their sum when
// renormalised.
//
// Bound by instruction issue and by the chain of dependent reductions, not by
// memory: 8192 x 256 logits (8.9 MB, 1.7 us at this card's copy rate) take 9.8 us,
// 64 x 256 take 4.9 us, launch included.
//
// LPT lanes hold a token's row; a lane owns V consecutive experts of one
// group (groups rounded up to a power of two of lane runs), so ascending
// lanes are ascending experts and ties fall to the lowest lane.  Scores are
// compared as order-preserving unsigned integers, 0 for an expert that cannot
// be chosen; everything stays in registers.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float sigmoidf(float x) { return 1.0f / (1.0f + expf(-x)); }

// A chosen expert's score up to a factor that all the chosen share, for
// renormalised weights: exp(x) sigmoid(-x) = sigmoid(x) over exp(ms), ms < 0 the largest
// of their logits, so that the ratios of scores below FP32's range are kept.
__device__ __forceinline__ float chosen_sigmoid(float x, float ms) {
    return ms < 0.0f ? expf(x - ms) * sigmoidf(-x) : sigmoidf(x);
}

// bits of the finite floats below -80: kLowLogits of them from kLowFirst on
constexpr uint32_t kLowFirst = 0xC2A00001u, kLowLogits = 0xFF800000u - kLowFirst;

constexpr int kMaxTopk = 16;

struct RouteArgs {
    int64_t T, ld;
    int E, topk, groups, gs, lpg, topk_groups, group_top, sigmoid, renorm, vec;
    float scale;
};

// V consecutive logits of a row from element `at` on (n of them exist; the others -inf)
template <int V, class T>
__device__ __forceinline__ void load_logits(const T* row, int at, int n, int vec, float (&v)[V]) {
    if (vec && n == V) {
        load_n<V>(row + at, v);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = j < n ? f32_of(row[at + j]) : kNegInf;
    }
}

template <class T, int LPT, int V>
__global__ __launch_bounds__(256) void route(const T* __restrict__ x, const float* __restrict__ bias, RouteArgs a,
                                             int32_t* __restrict__ idx, float* __restrict__ w) {
    __shared__ int chosen[256 / LPT][kMaxTopk];
    const int lane = threadIdx.x & 63, sl = lane & (LPT - 1), seg0 = lane & ~(LPT - 1), seg = threadIdx.x / LPT;
    const int64_t token = (int64_t(blockIdx.x) * 256 + threadIdx.x) / LPT;
    const bool there = token < a.T;
    const int g = sl / a.lpg, p = sl - g * a.lpg;
    const int left = a.gs - p * V, n = !there || g >= a.groups || left < 0 ? 0 : (left < V ? left : V);
    const int e0 = g * a.gs + p * V;
    const T* row = x + (there ? token : 0) * a.ld;
    float v[V], b[V];
    load_logits<V>(row, e0, n, a.vec, v);
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = bias && j < n ? bias[e0 + j] : 0.0f;
    if (sl < kMaxTopk) chosen[seg][sl] = -1;
    float m = 0.0f, inv = 0.0f;
    uint32_t key[V];
    if (a.sigmoid) {
        float s[V];
        uint32_t low = ~0u;            // below kLowLogits where a finite logit is below -80
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s[j] = sigmoid_fast(v[j]);
            const uint32_t u = __float_as_uint(v[j]) - kLowFirst;
            low = u < low ? u : low;
        }
        if (low < kLowLogits) {        // exp(x) down to FP32's smallest subnormal, where the reciprocal gives 0
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = v[j] < -80.0f ? expf(v[j]) : s[j];
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float c = s[j] + b[j];
            key[j] = (v[j] == kNegInf || c == kNegInf) ? 0u : ordered(c);
        }
    } else {
        m = kNegInf;
#pragma unroll
        for (int j = 0; j < V; ++j) m = fmaxf(m, v[j]);
        m = lanes_max<LPT>(m);
        if (m == kNegInf) m = 0.0f;
        float s[V], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) sum += s[j] = expf(v[j] - m);
        sum = lanes_sum<LPT>(sum);
        inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float c = s[j] * inv + b[j];
            key[j] = (v[j] == kNegInf || c == kNegInf) ? 0u : ordered(c);
        }
    }
    if (a.topk_groups < a.groups) {
        uint32_t k1 = 0, k2 = 0;       // the two largest keys of the lane, then of its group
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t lo = key[j] < k1 ? key[j] : k1;
            k1 = key[j] > k1 ? key[j] : k1;
            k2 = lo > k2 ? lo : k2;
        }
        for (int o = 1; o < a.lpg; o <<= 1) {
            const uint32_t t1 = __shfl_xor(k1, o, 64), t2 = __shfl_xor(k2, o, 64);
            const uint32_t lo = t1 < k1 ? t1 : k1, hi2 = t2 > k2 ? t2 : k2;
            k1 = t1 > k1 ? t1 : k1;
            k2 = lo > hi2 ? lo : hi2;
        }
        uint32_t gk = k1;
        if (a.group_top == 2 && k2 != 0) {
            const float sum = unordered(k1) + unordered(k2);
            gk = sum == kNegInf ? 1u : ordered(sum);
        }
        int rank = 0;
        for (int q = 0; q < a.groups; ++q) {
            const uint32_t o = __shfl(gk, seg0 + q * a.lpg, 64);
            rank += (o > gk || (o == gk && q < g)) ? 1 : 0;
        }
        if (rank >= a.topk_groups) {
#pragma unroll
            for (int j = 0; j < V; ++j) key[j] = 0u;
        }
    }
    // the chosen, one after the other: the segment's largest key belongs to its
    // lowest lane that holds it, there to the first element that equals it
    for (int i = 0; i < a.topk; ++i) {
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) best = key[j] > best ? key[j] : best;
        const uint32_t top = lanes_max<LPT>(best);
        uint64_t who = __builtin_amdgcn_ballot_w64(best == top && top != 0u);
        if (LPT < 64) who = (who >> seg0) & ((uint64_t(1) << (LPT & 63)) - 1);
        bool open = who != 0 && sl == int(__builtin_ctzll(who));
        int at = 0;
        const bool mine = open;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool hit = open && key[j] == best;
            key[j] = hit ? 0u : key[j];
            at = hit ? j : at;
            open = open && !hit;
        }
        if (mine) chosen[seg][i] = e0 + at;
    }
    __syncthreads();
    const int mine = there && sl < a.topk ? chosen[seg][sl] : -1;      // lane i < topk takes the i-th
    const float xs = mine >= 0 ? f32_of(row[mine]) : kNegInf;
    float wt;
    if (a.sigmoid) {
        const float ms = a.renorm ? lanes_max<LPT>(xs) : 0.0f;
        wt = mine >= 0 ? chosen_sigmoid(xs, ms) : 0.0f;
        if (a.renorm) {
            const float sum = lanes_sum<LPT>(wt);
            wt = sum > 0.0f ? wt / sum : 0.0f;
        }
    } else if (a.renorm) {             // a softmax over the chosen alone: relative to their own maximum
        const float ms = lanes_max<LPT>(xs);
        wt = mine >= 0 ? expf(xs - ms) : 0.0f;
        const float sum = lanes_sum<LPT>(wt);
        wt = sum > 0.0f ? wt / sum : 0.0f;
    } else {
        wt = mine >= 0 ? expf(xs - m) * inv : 0.0f;
    }
    if (there && sl < a.topk) {
        idx[token * a.topk + sl] = mine;
        w[token * a.topk + sl] = wt * a.scale;
    }
}

// The gradient of the logits.  With p_i = s_i / v (v the sum over the chosen)
// and d_i = sum_j (g_i - g_j) p_j, renormalised weights give
//   softmax dx_i = scale p_i d_i,   sigmoid dx_i = scale p_i (1 - s_i) d_i
// for the chosen and 0 for the others; otherwise sigmoid dx_i = scale g_i s_i
// (1 - s_i) and softmax dx_e = s_e (scale g_e [e chosen] - scale sum_j g_j s_j)
// for every expert.  The differences g_i - g_j keep a single renormalised
// weight's gradient exactly 0.
//
// LPT lanes hold a token's row, V experts each, in 16-byte pieces (U experts) that
// alternate over the lanes; where rows do not consist of such pieces, one by one (U
// = 1), neighbouring lanes on neighbouring experts.  Bound by instruction issue above
// launch: FP32 logits, sigmoid, us: 64 x 256 4.8, 8192 x 256 7.3, 14890 x 330 14.8 (with
// V consecutive experts per lane 5.1, 8.3, 19.8).
template <class T, int LPT, int V, int U>
__global__ __launch_bounds__(256) void route_backward(const T* __restrict__ x, const int32_t* __restrict__ idx,
                                                      const float* __restrict__ dw, RouteArgs a, T* __restrict__ dx) {
    const int lane = threadIdx.x & 63, sl = lane & (LPT - 1), seg0 = lane & ~(LPT - 1);
    const int64_t token = (int64_t(blockIdx.x) * 256 + threadIdx.x) / LPT;
    const bool there = token < a.T;
    const int64_t tk = there ? token : 0;
    const T* row = x + tk * a.ld;
    const auto expert = [&](int j) { return (j / U * LPT + sl) * U + j % U; };
    const bool dense = !a.sigmoid && !a.renorm;
    float v[V], m = 0.0f, inv = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = 0.0f;
    if (dense) {
        m = kNegInf;
#pragma unroll
        for (int j = 0; j < V; j += U) {
            float p[U];
#pragma unroll
            for (int u = 0; u < U; ++u) p[u] = kNegInf;
            if (there && expert(j) < a.E) {
                if constexpr (U > 1)
                    load_n<U>(row + expert(j), p);
                else
                    p[0] = f32_of(row[expert(j)]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) m = fmaxf(m, v[j + u] = p[u]);
        }
        m = lanes_max<LPT>(m);
        if (m == kNegInf) m = 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) sum += expf(v[j] - m);
        sum = lanes_sum<LPT>(sum);
        inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    }
    int mine = -1;
    float g = 0.0f;
    if (there && sl < a.topk) {
        mine = idx[token * a.topk + sl];
        if (mine >= a.E) mine = -1;
        if (mine >= 0) g = dw[token * a.topk + sl] * a.scale;
    }
    const float xs = mine >= 0 ? f32_of(row[mine]) : kNegInf;
    float c = 0.0f, D = 0.0f;          // the chosen expert's own term; the sum over the chosen
    if (a.renorm) {
        const float ms = lanes_max<LPT>(xs);
        float p = mine < 0 ? 0.0f : a.sigmoid ? chosen_sigmoid(xs, ms) : expf(xs - ms);
        const float sum = lanes_sum<LPT>(p);
        p = sum > 0.0f ? p / sum : 0.0f;
        float d = 0.0f;
        for (int j = 0; j < a.topk; ++j) {
            const float gj = __shfl(g, seg0 + j, 64), pj = __shfl(p, seg0 + j, 64);
            d += (g - gj) * pj;
        }
        c = p * d;
        if (a.sigmoid && mine >= 0) c *= sigmoidf(-xs);
    } else if (a.sigmoid) {
        c = mine >= 0 ? g * sigmoidf(xs) * sigmoidf(-xs) : 0.0f;
    } else {
        c = mine >= 0 ? g * (expf(xs - m) * inv) : 0.0f;
        D = lanes_sum<LPT>(c);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = dense ? -(expf(v[j] - m) * inv) * D : 0.0f;
    for (int i = 0; i < a.topk; ++i) {
        const int e = __shfl(mine, seg0 + i, 64);
        const float ci = __shfl(c, seg0 + i, 64);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] += expert(j) == e ? ci : 0.0f;
    }
    T* out = dx + tk * a.E;
#pragma unroll
    for (int j = 0; j < V; j += U) {
        if (!there || expert(j) >= a.E) continue;
        if constexpr (U > 1) {
            float p[U];
#pragma unroll
            for (int u = 0; u < U; ++u) p[u] = v[j + u];
            store_n<U>(out + expert(j), p);
        } else {
            store1(out + expert(j), v[j]);
        }
    }
}

// ---------------------------------------------------------------------------
// The row of every (token, choice) of the local experts first .. first + G - 1,
// in the order of the entries (stable, no atomics on the result), the experts'
// counts and, in the contiguous layout (m_max = 0), their offsets rounded up
// to 128 rows; in the masked layout expert g owns rows g m_max .. and entries
// past m_max have no row.
//
// One workgroup per `chunk` entries.  It counts every expert's entries before
// its chunk and in all (32 counters per expert, so that at most two lanes of a
// wave, l and l + 32, meet on an address; 32 entries per thread in flight), then ranks its own chunk 1024 entries at a time: the lanes of a wave
// with the same expert find each other with one ballot per bit of the index,
// the waves' counts are summed in order.  No workgroup waits for another, at the
// price of each reading every entry: 65536 entries take 9.8 us (64 workgroups).
constexpr int kMaxLocal = 256;

__global__ __launch_bounds__(1024) void rows_layout(const int32_t* __restrict__ idx, int64_t n, int first, int G,
                                                    int64_t chunk, int64_t m_max, int32_t* __restrict__ row_of,
                                                    int32_t* __restrict__ offsets, int32_t* __restrict__ counts) {
    __shared__ uint32_t hist[kMaxLocal * 32];
    __shared__ uint32_t wave_count[16][kMaxLocal];
    __shared__ uint32_t base[kMaxLocal];       // rows of the expert before the current entry
    __shared__ uint32_t start[kMaxLocal + 1];  // first row of the expert
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t lo = int64_t(blockIdx.x) * chunk, hi = lo + chunk < n ? lo + chunk : n;
    for (int i = t; i < G * 32; i += 1024) hist[i] = 0;
    __syncthreads();
    auto add = [&](int32_t id) {
        const uint32_t e = uint32_t(id) - uint32_t(first);
        if (e < uint32_t(G)) atomicAdd(&hist[e * 32 + (lane & 31)], 1u);
    };
    // entries [from, to), from a multiple of 1024
    auto count = [&](int64_t from, int64_t to) {
        int64_t i = from + 4 * t;
        typedef int i32x4 __attribute__((ext_vector_type(4)));
        for (; i + 7 * 4096 + 4 <= to; i += 8 * 4096) {
            i32x4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = ld<i32x4>(idx + i + 4096 * k);
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) add(v[k][j]);
        }
#pragma unroll 4
        for (; i + 4 <= to; i += 4096) {
            const i32x4 v = ld<i32x4>(idx + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) add(v[j]);
        }
        for (int64_t j = i; j < to && j < i + 4; ++j) add(idx[j]);
        __syncthreads();
    };
    auto total = [&](int e) {
        uint32_t c = 0;
#pragma unroll 8
        for (int i = 0; i < 32; ++i) c += hist[e * 32 + ((i + e) & 31)];
        return c;
    };
    if (lo > 0) count(0, lo);
    if (t < G) base[t] = lo > 0 ? total(t) : 0u;
    __syncthreads();
    count(lo, n);
    if (t < kMaxLocal) {
        const uint32_t c = t < G ? total(t) : 0u;
        if (blockIdx.x == 0 && t < G) counts[t] = int32_t(m_max && c > uint64_t(m_max) ? uint32_t(m_max) : c);
        // first rows: an inclusive scan over the wave's 64 experts, the four waves' sums below
        uint32_t sum = m_max ? uint32_t(m_max) : (c + 127u) / 128u * 128u;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t below = __shfl_up(sum, o, 64);
            sum += lane >= o ? below : 0u;
        }
        start[t + 1] = sum;
    }
    if (t == 0) start[0] = 0;
    __syncthreads();
    uint32_t below = 0;
    if (t < kMaxLocal)
        for (int w = 0; w < wave; ++w) below += start[64 * w + 64];
    __syncthreads();
    if (t < kMaxLocal) start[t + 1] += below;
    __syncthreads();
    if (blockIdx.x == 0 && offsets && t <= G) offsets[t] = int32_t(start[t]);
    for (int64_t at = lo; at < hi; at += 1024) {
        for (int i = t; i < 16 * kMaxLocal; i += 1024) wave_count[i / kMaxLocal][i % kMaxLocal] = 0;
        const int64_t i = at + t;
        const uint32_t e0 = i < hi ? uint32_t(idx[i]) - uint32_t(first) : uint32_t(G);
        const bool mine = e0 < uint32_t(G);
        const uint32_t e = mine ? e0 : uint32_t(G);
        __syncthreads();
        uint64_t same = ~uint64_t(0);
        for (int b = 0; (1 << b) <= G; ++b) {
            const uint64_t set = __builtin_amdgcn_ballot_w64((e >> b) & 1);
            same &= ((e >> b) & 1) ? set : ~set;
        }
        const uint32_t before = uint32_t(__builtin_popcountll(same & ((uint64_t(1) << lane) - 1)));
        if (mine && before == 0) wave_count[wave][e] = uint32_t(__builtin_popcountll(same));
        __syncthreads();
        if (t < G) {
            uint32_t run = base[t];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const uint32_t c = wave_count[k][t];
                wave_count[k][t] = run;
                run += c;
            }
            base[t] = run;
        }
        __syncthreads();
        if (i < hi) {
            int32_t row = -1;
            if (mine) {
                const uint32_t rank = wave_count[wave][e] + before;
                if (!m_max || rank < uint64_t(m_max)) row = int32_t(start[e] + rank);
            }
            row_of[i] = row;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// A token's row quantized 1x128 and written to its rows.  A wave takes 512
// channels of one token: eight per lane, 16 lanes to a 128-group, so one store
// instruction writes 512 bytes of a row.  Reading each token once and writing its
// codes k times moves 602 MB for 8192 tokens x 7168 channels x 8 rows; a row by row gather
// would read (and quantize) each token eight times.  Bound by the writes: 130 us,
// 4.6 TB/s against 5.2 for a plain copy; the scales' scattered 4-byte writes
// are the difference (with plain stores, 146 us with them and 121 without).  With
// 16 channels per lane the whole call takes (us, 16 / 8) 143 / 141 there, 180 / 170 from
// FP32 tokens, 25.4 / 27.4 for 1024 tokens, 34.5 / 32.6 for 20000 tokens x 512 channels x 6.
constexpr int kChan = 8, kWaveChan = 64 * kChan, kLanes = kBlock / kChan;      // kLanes: lanes of a 128-group

struct RowsOut {
    uint8_t* q;
    float* s;
    int64_t H, kbs, rows_per;      // rows_per: rows of one scale array (M_total, or M_max of an expert)
    template <bool MASKED>
    __device__ __forceinline__ float* scale(uint32_t row, uint32_t kb) const {
        if (!MASKED) return s + kb * rows_per + row;
        const uint32_t b = row / uint32_t(rows_per);
        return s + (b * kbs + kb) * rows_per + (row - b * uint32_t(rows_per));
    }
};

// Workgroup b of n runs on XCD b mod 8; it takes item x (n / 8) + b / 8, so
// that an XCD works through consecutive tokens: their rows' scales, four bytes
// at a time beside those of the expert's previous rows, fill whole lines of
// one L2.  A bijection on [0, n).
constexpr uint32_t kXcds = 8;
__device__ __forceinline__ uint32_t xcd_run(uint32_t b, uint32_t n) {
    const uint32_t per = n / kXcds;
    return b < per * kXcds ? (b % kXcds) * per + b / kXcds : b;
}

// zero rows [counts[g], padded count) of every expert: wave p = (expert, row)
__device__ __forceinline__ void zero_padding(uint32_t p, const int32_t* offsets, const int32_t* counts, int64_t R,
                                             const RowsOut& o, int lane) {
    const uint32_t g = p / 127;
    const int64_t row = int64_t(offsets[g]) + counts[g] + p % 127;
    if (row < 0 || row >= offsets[g + 1] || row >= R) return;
    for (int64_t c = lane * 16; c < o.H; c += 1024) st<u32x4>(o.q + row * o.H + c, u32x4{0u, 0u, 0u, 0u});
    for (int64_t kb = lane; kb < o.kbs; kb += 64) *o.scale<false>(uint32_t(row), uint32_t(kb)) = 0.0f;
}

template <class T, bool MASKED, bool STREAM>
__global__ __launch_bounds__(256) void dispatch_rows(const T* __restrict__ x, const int32_t* __restrict__ row_of,
                                                     uint32_t waves, int topk, uint32_t chunks, uint32_t blocks,
                                                     RowsOut o, const int32_t* __restrict__ offsets,
                                                     const int32_t* __restrict__ counts, uint32_t G, int64_t R) {
    const int lane = threadIdx.x & 63;
    const uint32_t b = blockIdx.x < blocks ? xcd_run(blockIdx.x, blocks) : blockIdx.x;
    const uint32_t w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + b * 4;
    if (b >= blocks) {
        const uint32_t p = w - blocks * 4;
        if (!MASKED && p < 127 * G) zero_padding(p, offsets, counts, R, o, lane);
        return;
    }
    if (w >= waves) return;
    const uint32_t token = w / chunks, c = w - token * chunks;
    const uint32_t ch = c * kWaveChan + lane * kChan;
    float v[kChan];
#pragma unroll
    for (int i = 0; i < kChan; ++i) v[i] = 0.0f;
    const int32_t* rows = row_of + int64_t(token) * topk;
    int32_t none = -1;
    for (int j = 0; j < topk; ++j) none &= rows[j];
    if (none < 0) return;                                // every entry elsewhere (-1): the token is not read
    if (ch < o.H) load_n<kChan, true>(x + int64_t(token) * o.H + ch, v);
    float sc;
    const auto code = encode_lane<typename encoder_of<T>::type>(v, sc);
    if (ch < o.H)
        for (int j = 0; j < topk; ++j) {
            const int64_t r = rows[j];
            if (r >= 0) st_out<STREAM>(o.q + r * o.H + ch, code);
        }
    const uint32_t kb = c * (64 / kLanes) + lane / kLanes;
    if (kb < o.kbs)
        for (int j = lane % kLanes; j < topk; j += kLanes) {
            const int32_t r = rows[j];
            if (r >= 0) *o.scale<MASKED>(uint32_t(r), kb) = sc;
        }
}

// ---------------------------------------------------------------------------
// The row layout and the rows themselves in one launch, for few entries: every
// workgroup counts all entries for itself, so none waits for another.  A
// workgroup takes four 512-channel chunks of one token; in the contiguous layout
// kPadParts more per expert clear its padding rows.  Bound by latency: 128 tokens x 8 entries,
// 7168 channels, 4.9 us against 3.9 + 3.7 us for the two launches it replaces.  The
// padding is most of a small contiguous call: with 1 / 8 / 16 parts, 1 token x 2 rows of 7168
// channels in 8 experts 13.7 / 4.5 / 4.0 us, 64 tokens x 8 in 32 experts 16.0 / 9.3 / 9.1.
//
// Up to 2048 entries, and up to about as many workgroups as the chip holds at once (256
// CUs x 8): each counts all entries, so more of them cost more than the second launch
// (us, one launch / two; tokens x channels x choices in 8 to 32 experts).  Contiguous: 256 x 7168 x 8
// (1024 workgroups) 11.7 / 14.2, 1024 x 512 x 2 6.8 / 7.6, 400 x 7168 x 4 (1600) 9.5 / 11.3, 2000 x
// 1024 x 1 10.1 / 8.0, 512 x 7168 x 2 (2048) 11.1 / 9.5, 1024 x 7168 x 2 (4096) 19.6 / 13.3, 2048 x
// 7168 x 1 (8192) 32.8 / 17.6; 512 x 7168 x 8 (4096 entries) 19.2 / 17.5.  Masked: 512 x 7168 x 2
// 7.1 / 9.1, 1024 x 4096 x 1 6.7 / 8.5, 2000 x 1024 x 1 8.6 / 8.2, 1500 x 7168 x 1 (6000) 17.9 / 14.0.
constexpr int64_t kSmallEntries = 2048;
template <bool MASKED>
constexpr int64_t small_grid() {
    return MASKED ? 2048 : 1600;
}
constexpr uint32_t kPadParts = 8;

template <class T, bool MASKED>
__global__ __launch_bounds__(256) void dispatch_small(const T* __restrict__ x, const int32_t* __restrict__ idx,
                                                      uint32_t tokens, int topk, uint32_t per_token, int first,
                                                      uint32_t G, RowsOut o, int32_t* __restrict__ row_of,
                                                      int32_t* __restrict__ offsets, int32_t* __restrict__ counts) {
    __shared__ uint32_t all[kMaxLocal], before[kMaxLocal], start[kMaxLocal + 1];
    const uint32_t t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const uint32_t token = blockIdx.x / per_token, part = blockIdx.x - token * per_token;
    const bool padding = token >= tokens;               // (uniform) the p-th of the padding's workgroups
    const uint32_t n = tokens * uint32_t(topk), mine = padding ? 0u : token * uint32_t(topk);
    const uint32_t c = part * 4 + wave, ch = c * kWaveChan + lane * kChan;
    float v[kChan];
#pragma unroll
    for (int i = 0; i < kChan; ++i) v[i] = 0.0f;
    if (!padding && ch < o.H) load_n<kChan, true>(x + int64_t(token) * o.H + ch, v);
    all[t] = before[t] = 0;                             // kMaxLocal threads
    __syncthreads();
    for (uint32_t i = t; i < n; i += 256) {
        const uint32_t e = uint32_t(idx[i]) - uint32_t(first);
        if (e < G) {
            atomicAdd(&all[e], 1u);
            if (i < mine) atomicAdd(&before[e], 1u);
        }
    }
    __syncthreads();
    if (!MASKED) {
        uint32_t sum = (all[t] + 127u) / 128u * 128u;
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) {
            const uint32_t below = __shfl_up(sum, k, 64);
            sum += int(lane) >= k ? below : 0u;
        }
        start[t + 1] = sum;
        if (t == 0) start[0] = 0;
        __syncthreads();
        uint32_t below = 0;
        for (uint32_t w = 0; w < wave; ++w) below += start[64 * w + 64];
        __syncthreads();
        start[t + 1] += below;
        __syncthreads();
        if (blockIdx.x == 0)
            for (uint32_t i = t; i <= G; i += 256) offsets[i] = int32_t(start[i]);
    }
    if (blockIdx.x == 0 && t < G) counts[t] = int32_t(MASKED && all[t] > uint64_t(o.rows_per) ? uint32_t(o.rows_per) : all[t]);
    if (padding) {
        const uint32_t p = blockIdx.x - tokens * per_token, g = p / kPadParts;
        for (uint32_t row = start[g] + all[g] + p % kPadParts * 4 + wave; row < start[g + 1]; row += kPadParts * 4) {
            for (int64_t i = lane * 16; i < o.H; i += 1024) st<u32x4>(o.q + int64_t(row) * o.H + i, u32x4{0u, 0u, 0u, 0u});
            for (uint32_t kb = lane; kb < o.kbs; kb += 64) *o.scale<false>(row, kb) = 0.0f;
        }
        return;
    }
    // lane j < topk: the row of the token's j-th entry
    int32_t row = -1;
    const uint32_t e = lane < uint32_t(topk) ? uint32_t(idx[mine + lane]) - uint32_t(first) : G;
    uint32_t rank = e < G ? before[e] : 0u;
    for (int j = 0; j < topk; ++j) rank += uint32_t(j) < lane && uint32_t(__builtin_amdgcn_readlane(int(e), j)) == e ? 1u : 0u;
    if (e < G && (!MASKED || rank < uint64_t(o.rows_per))) row = int32_t(MASKED ? e * uint32_t(o.rows_per) + rank : start[e] + rank);
    if (part == 0 && wave == 0 && lane < uint32_t(topk)) row_of[mine + lane] = row;
    float sc;
    const auto code = encode_lane<typename encoder_of<T>::type>(v, sc);
    for (int j = 0; j < topk; ++j) {
        const int64_t r = __builtin_amdgcn_readlane(row, j);
        if (r >= 0 && ch < o.H) st_out<false>(o.q + r * o.H + ch, code);
    }
    const uint32_t kb = c * (64 / kLanes) + lane / kLanes;
    for (int j0 = 0; j0 < topk; j0 += kLanes) {
        const int32_t r = __shfl(row, j0 + int(lane % kLanes), 64);      // lanes from topk on hold -1
        if (r >= 0 && kb < o.kbs) *o.scale<MASKED>(uint32_t(r), kb) = sc;
    }
}

// ---------------------------------------------------------------------------
// out_t = sum_j w_tj y[row_tj], in the order of the choices, in FP32.  A wave
// takes 512 channels of one token, eight per lane (many FP32 rows:
// four, one 16-byte load).  Bound by the reads: 8192
// tokens x 8 rows of 7168 BF16 channels, 1.06 GB, 178 us, 5.9 TB/s (the rows are read once: with the
// non-temporal hint, without it 204 us).
template <class TY, class TO, int V>
__global__ __launch_bounds__(256) void combine(const TY* __restrict__ y, int64_t R, int64_t H,
                                               const int32_t* __restrict__ row_of, const float* __restrict__ wts,
                                               uint32_t waves, int topk, uint32_t chunks, TO* __restrict__ out) {
    const int lane = threadIdx.x & 63;
    const uint32_t w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + blockIdx.x * 4;
    if (w >= waves) return;
    const uint32_t token = w / chunks, ch = (w - token * chunks) * (64 * V) + lane * V;
    if (ch >= H) return;
    const int32_t* rows = row_of + int64_t(token) * topk;
    const float* wt = wts ? wts + int64_t(token) * topk : nullptr;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    // four entries at a time, their loads in flight together.  Measured (us, one
    // at a time / four): 64 tokens of 7168 channels x 8 rows 4.9 / 4.4, 512 11.6 /
    // 11.3, 8192 182.2 / 183.0.
    for (int j0 = 0; j0 < topk; j0 += 4) {
        bool has[4];
        Raw<TY, V> v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = j0 + j < topk ? rows[j0 + j] : -1;
            has[j] = r >= 0 && r < R;
            if (has[j]) v[j].template load<true>(y + r * H + ch);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (has[j]) {
                const float f = wt ? wt[j0 + j] : 1.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(f, v[j].get(i), acc[i]);
            }
        }
    }
    store_n<V>(out + int64_t(token) * H + ch, acc);
}

// ---------------------------------------------------------------------------
// The backward pass of combine: dw_tj = <dout_t, y[row_tj]> in FP32, and the
// rows dy = w_tj Q(dout_t), where Q is the 1x128 quantization of dout_t: every
// row of a token shares its codes, and its scales are |w| times the token's
// (the sign of w goes into the codes).  A workgroup per token; a wave takes 512
// channels at a time, eight per lane (V), and F entries' rows in flight.  Bound by memory:
// 3001 tokens x 8 rows of 7168 BF16 channels, 565 MB, 112 us, 5.0 TB/s (16
// channels per lane: 118 us).
//
// Waves of a workgroup: at most 4 for streaming outputs, 8 otherwise, 16 with four
// entries in flight for few tokens, whose time is that of one workgroup; evenly loaded.
// Measured (us, 4 / 8 / 16, 7168 channels x 8 rows in BF16 unless noted): 64 tokens 21.9 /
// 15.6 / 11.0, 256 tokens 32.5 / 22.3 / 16.7; 512 tokens of 4096 channels 20.6 / 14.5 / 16.0, 512
// tokens x 2 rows 11.5 / 9.0 / 11.9; 1024 tokens (streaming) 43.9 / 48.2 / 51.7, 3001 tokens
// 112.4 / 115.2 / 140.5.
constexpr int64_t kFewTokens = 256;

// Channels of a lane.  Many FP32 rows: four, one 16-byte load (us, eight / four: 1024 tokens x 8
// rows of 7168 channels 69.2 / 66.8, 3001 199 / 178, 8192 568 / 516; 512 tokens, not
// streaming, 12.8 / 14.4).
template <class TY, bool STREAM>
constexpr int back_run() {
    return STREAM && sizeof(TY) == 4 ? 4 : 8;
}
template <class TD, class TY, bool STREAM, int F>
__global__ __launch_bounds__(1024) void combine_backward(const TD* __restrict__ dout, const TY* __restrict__ y,
                                                           const int32_t* __restrict__ row_of,
                                                           const float* __restrict__ wts, int64_t T_, int topk, RowsOut o,
                                                           const int32_t* __restrict__ offsets,
                                                           const int32_t* __restrict__ counts, int64_t G, int64_t R,
                                                           float* __restrict__ dw) {
    constexpr int V = back_run<TY, STREAM>(), kGroup = kBlock / V;            // channels of a lane, lanes of a 128-group
    __shared__ float part[16][kMaxTopk];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    if (blockIdx.x >= T_) {
        const int64_t p = (int64_t(blockIdx.x) - T_) * waves + wave;
        if (p < 127 * G) zero_padding(uint32_t(p), offsets, counts, R, o, lane);
        return;
    }
    const int64_t token = xcd_run(blockIdx.x, uint32_t(T_));
    const int32_t* rows = row_of + token * topk;
    const float* wt = wts + token * topk;
    float dot[kMaxTopk];
#pragma unroll
    for (int j = 0; j < kMaxTopk; ++j) dot[j] = 0.0f;
    const uint32_t chunks = uint32_t((o.H + 64 * V - 1) / (64 * V));
    for (uint32_t c = wave; c < chunks; c += waves) {
        const uint32_t ch = c * (64 * V) + lane * V;
        const bool in = ch < o.H;
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.0f;
        if (in) load_n<V>(dout + token * o.H + ch, v);
        float sc;
        const auto code = encode_lane<typename encoder_of<TD>::type>(v, sc);
        const uint32_t kb = c * (64 / kGroup) + lane / kGroup;
#pragma unroll
        for (int j0 = 0; j0 < kMaxTopk; j0 += F) {
            if (j0 < topk) {
                int64_t r[F];
                Raw<TY, V> u[F];
#pragma unroll
                for (int j = 0; j < F; ++j) {
                    r[j] = j0 + j < topk && in ? rows[j0 + j] : -1;
                    if (r[j] >= R) r[j] = -1;
                    if (r[j] >= 0) u[j].template load<STREAM>(y + r[j] * o.H + ch);
                }
#pragma unroll
                for (int j = 0; j < F; ++j) {
                    if (r[j] >= 0) {
                        const float wj = wt[j0 + j];
                        const uint32_t flip = wj < 0.0f ? 0x80808080u : 0u;
                        auto signed_code = code;
#pragma unroll
                        for (int i = 0; i < V / 4; ++i) signed_code[i] ^= flip;
                        st_out<STREAM>(o.q + r[j] * o.H + ch, signed_code);
                        if (lane % kGroup == 0) *o.scale<false>(uint32_t(r[j]), kb) = sc * fabsf(wj);
#pragma unroll
                        for (int i = 0; i < V; ++i) dot[j0 + j] = fmaf(v[i], u[j].get(i), dot[j0 + j]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kMaxTopk; ++j) {
        dot[j] = lanes_sum<64>(dot[j]);
        if (lane == 0) part[wave][j] = dot[j];
    }
    __syncthreads();
    const int j = threadIdx.x;
    if (j < topk) {
        float sum = 0.0f;
        for (int k = 0; k < waves; ++k) sum += part[k][j];
        dw[token * topk + j] = sum;
    }
}

// ---------------------------------------------------------------------------
// host

inline int pow2_at_least(int64_t n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

template <class T, int LPT, int V>
hipError_t run_route(const void* x, const float* bias, const RouteArgs& a, int32_t* idx, float* w, hipStream_t stream) {
    const int64_t blocks = (a.T + 256 / LPT - 1) / (256 / LPT);
    return launch_kernel(route<T, LPT, V>, dim3(unsigned(blocks)), dim3(256), stream, static_cast<const T*>(x), bias, a, idx, w);
}
template <class T, int LPT, int V>
hipError_t run_route_backward(const void* x, const int32_t* idx, const float* dw, const RouteArgs& a, void* dx,
                              hipStream_t stream) {
    const int64_t blocks = (a.T + 256 / LPT - 1) / (256 / LPT);
    constexpr int U = 16 / int(sizeof(T)) < V ? 16 / int(sizeof(T)) : V;
    const bool pieces = a.ld % U == 0 && a.E % U == 0;
    return launch_kernel(pieces ? route_backward<T, LPT, V, U> : route_backward<T, LPT, V, 1>, dim3(unsigned(blocks)), dim3(256), stream, static_cast<const T*>(x), idx, dw, a, static_cast<T*>(dx));
}

}  // namespace moe_detail

using namespace moe_detail;

hipError_t launch_route(const RouteCall& c, hipStream_t stream) {
    RouteArgs a{c.T, c.ld, int(c.E), int(c.topk), int(c.n_groups), int(c.E / c.n_groups), 0, int(c.topk_groups), c.group_top,
                c.sigmoid, c.renorm, 0, c.scale};
    const int ng = pow2_at_least(c.n_groups);
    const int el = c.bf16 ? 2 : 4;
    // 16 lanes per token (four tokens per wave) or the whole wave.  The wave's
    // chain is shorter (fewer experts per lane), the 16 lanes' instructions per
    // token fewer.  Measured (us, 16 lanes / 64): 256 experts 7.8 / 4.9 at 64 tokens, 8.3 / 6.7 at
    // 4096, 10.7 / 9.8 at 8192, 15.2 / 16.3 at 16384; 128 experts 6.4 / 8.0 at 8192;
    // 64 experts 3.7 / 4.1 at 64, 4.5 / 8.1 at 8192.
    const int share = (a.gs + 16 / ng - 1) / (16 / ng);      // experts per lane of 16
    const int lpt = share > 16 || (share > 8 && c.T <= 8192) || (share > 4 && c.T <= 4096) ? 64 : 16;
    a.lpg = lpt / ng;
    const int need = (a.gs + a.lpg - 1) / a.lpg, v = need <= 4 ? 4 : need <= 8 ? 8 : 16;
    const int unit = v * el < 16 ? v * el : 16;
    a.vec = (c.ld * el) % unit == 0 && (int64_t(a.gs) * el) % unit == 0;
#define FP8FG_ROUTE(T, L, V) \
    if (lpt == L && v == V) return run_route<T, L, V>(c.x, c.bias, a, c.idx, c.w, stream);
#define FP8FG_ROUTES(T) \
    FP8FG_ROUTE(T, 16, 4) FP8FG_ROUTE(T, 16, 8) FP8FG_ROUTE(T, 16, 16) FP8FG_ROUTE(T, 64, 4) FP8FG_ROUTE(T, 64, 8) FP8FG_ROUTE(T, 64, 16)
    if (c.bf16) {
        FP8FG_ROUTES(uint16_t)
    } else {
        FP8FG_ROUTES(float)
    }
    return hipErrorInvalidValue;
}

hipError_t launch_route_backward(const RouteCall& c, const float* dw, void* dx, hipStream_t stream) {
    RouteArgs a{c.T, c.ld, int(c.E), int(c.topk), 1, int(c.E), 0, 1, 1, c.sigmoid, c.renorm, 0, c.scale};
    // 16 lanes of 32 experts each for up to 512 are slower (us, 64 x 8 / 16 x 32): 1000 x 330 4.1 /
    // 5.6, 16384 x 512 softmax 19.7 / 21.5
    const int lpt = c.E <= 256 ? 16 : 64;
    const int need = (a.E + lpt - 1) / lpt, v = need <= 4 ? 4 : need <= 8 ? 8 : 16;
#define FP8FG_ROUTE_B(T, L, V) \
    if (lpt == L && v == V) return run_route_backward<T, L, V>(c.x, c.idx, dw, a, dx, stream);
#define FP8FG_ROUTES_B(T) \
    FP8FG_ROUTE_B(T, 16, 4) FP8FG_ROUTE_B(T, 16, 8) FP8FG_ROUTE_B(T, 16, 16) FP8FG_ROUTE_B(T, 64, 8) FP8FG_ROUTE_B(T, 64, 16)
    if (c.bf16) {
        FP8FG_ROUTES_B(uint16_t)
    } else {
        FP8FG_ROUTES_B(float)
    }
    return hipErrorInvalidValue;
}

static hipError_t launch_rows_layout(const int32_t* idx, int64_t n, int64_t first, int64_t G, int64_t m_max, int32_t* row_of,
                              int32_t* offsets, int32_t* counts, hipStream_t stream) {
    int64_t chunk = 1024, blocks = (n + chunk - 1) / chunk;
    if (blocks > 256) {
        chunk = (n + 256 * 1024 - 1) / (256 * 1024) * 1024;
        blocks = (n + chunk - 1) / chunk;
    }
    if (blocks == 0) blocks = 1;       // no entries: the counts and offsets are still written
    return launch_kernel(rows_layout, dim3(unsigned(blocks)), dim3(1024), stream, idx, n, int(first), int(G), chunk, m_max,
                         row_of, offsets, counts);
}

template <class T, bool MASKED>
static hipError_t run_dispatch(const void* x, int64_t T_, const int32_t* idx, int64_t topk, int64_t first, int64_t G,
                               int64_t R, const RowsOut& o, int32_t* row_of, int32_t* offsets, int32_t* counts,
                               hipStream_t stream) {
    const int64_t n = T_ * topk, chunks = (o.H + kWaveChan - 1) / kWaveChan, waves = T_ * chunks;
    const int64_t per_token = (chunks + 3) / 4;
    if (n <= kSmallEntries && waves > 0 && T_ * per_token <= small_grid<MASKED>()) {
        const int64_t grid = T_ * per_token + (MASKED ? 0 : G * kPadParts);
        return launch_kernel(dispatch_small<T, MASKED>, dim3(unsigned(grid)), dim3(256), stream, static_cast<const T*>(x),
                             idx, uint32_t(T_), int(topk), uint32_t(per_token), int(first), uint32_t(G), o, row_of,
                             offsets, counts);
    }
    const int64_t blocks = (waves + 3) / 4, grid = blocks + (MASKED ? 0 : (127 * G + 3) / 4);
    if (!grid_fits(grid, 256)) return hipErrorInvalidConfiguration;      // before the first of the two launches
    const hipError_t e = launch_rows_layout(idx, n, first, G, MASKED ? o.rows_per : 0, row_of, offsets, counts, stream);
    if (e != hipSuccess || waves == 0) return e;
    // (R rows bound what is written: the routing is known on the device only)
    const bool stream_out = (R < n ? R : n) * o.H >= kStreamBytes;
    return launch_kernel(stream_out ? dispatch_rows<T, MASKED, true> : dispatch_rows<T, MASKED, false>,
                         dim3(unsigned(grid)), dim3(256), stream, static_cast<const T*>(x), row_of, uint32_t(waves),
                         int(topk), uint32_t(chunks), uint32_t(blocks), o, offsets, counts, uint32_t(G), R);
}

hipError_t launch_dispatch(const void* x, int bf16, int64_t T, int64_t H, const int32_t* idx, int64_t topk,
                           int64_t first, int64_t G, int64_t R, int64_t m_max, uint8_t* q, float* s, int32_t* row_of,
                           int32_t* offsets, int32_t* counts, hipStream_t stream) {
    const RowsOut o{q, s, H, (H + kBlock - 1) / kBlock, m_max ? m_max : R};
    if (m_max)
        return bf16 ? run_dispatch<uint16_t, true>(x, T, idx, topk, first, G, R, o, row_of, nullptr, counts, stream)
                    : run_dispatch<float, true>(x, T, idx, topk, first, G, R, o, row_of, nullptr, counts, stream);
    return bf16 ? run_dispatch<uint16_t, false>(x, T, idx, topk, first, G, R, o, row_of, offsets, counts, stream)
                : run_dispatch<float, false>(x, T, idx, topk, first, G, R, o, row_of, offsets, counts, stream);
}

template <class TY, class TO>
static hipError_t run_combine(const void* y, int64_t R, int64_t H, const int32_t* row_of, const float* w, int64_t T,
                              int64_t topk, void* out, hipStream_t stream) {
    // FP32 rows of 32 MB and more: four channels per lane.  Measured (us, eight / four): 64
    // tokens x 8 rows of 7168 channels 5.7 / 6.9, 500 x 8 x 2048 (32 MB) 8.7 / 8.8, 1024 x 8 x
    // 7168 50.3 / 44.8, 8192 x 8 x 7168 395 / 341.
    const bool four = sizeof(TY) == 4 && T * topk * H * 4 >= kStreamBytes;
    const int64_t per = 64 * (four ? 4 : 8), chunks = (H + per - 1) / per, blocks = (T * chunks + 3) / 4;
    auto* kernel = combine<TY, TO, 8>;
    if constexpr (sizeof(TY) == 4)
        if (four) kernel = combine<TY, TO, 4>;
    return launch_kernel(kernel, dim3(unsigned(blocks)), dim3(256), stream, static_cast<const TY*>(y), R, H, row_of, w,
                         uint32_t(T * chunks), int(topk), uint32_t(chunks), static_cast<TO*>(out));
}

hipError_t launch_combine(const void* y, int y_bf16, int64_t R, int64_t H, const int32_t* row_of, const float* w,
                          int64_t T, int64_t topk, void* out, int out_fp32, hipStream_t stream) {
    if (y_bf16)
        return out_fp32 ? run_combine<uint16_t, float>(y, R, H, row_of, w, T, topk, out, stream)
                        : run_combine<uint16_t, uint16_t>(y, R, H, row_of, w, T, topk, out, stream);
    return out_fp32 ? run_combine<float, float>(y, R, H, row_of, w, T, topk, out, stream)
                    : run_combine<float, uint16_t>(y, R, H, row_of, w, T, topk, out, stream);
}

template <class TD, class TY>
static hipError_t run_combine_backward(const void* dout, int64_t T, int64_t H, const void* y, int64_t R,
                                       const int32_t* row_of, const float* w, int64_t topk, const int32_t* offsets,
                                       const int32_t* counts, int64_t G, uint8_t* q, float* s, float* dw,
                                       hipStream_t stream) {
    const RowsOut o{q, s, H, (H + kBlock - 1) / kBlock, R};
    const bool stream_out = (R < T * topk ? R : T * topk) * H >= kStreamBytes, few = T <= kFewTokens && !stream_out;
    const int64_t per = 64 * (stream_out ? back_run<TY, true>() : back_run<TY, false>()), chunks = (H + per - 1) / per;
    const int64_t most = few ? 16 : stream_out ? 4 : 8, each = (chunks + most - 1) / most;
    const int64_t waves = chunks ? (chunks + each - 1) / each : 1;
    auto* kernel = few          ? combine_backward<TD, TY, false, 4>
                   : stream_out ? combine_backward<TD, TY, true, 1>
                                : combine_backward<TD, TY, false, 1>;
    return launch_kernel(kernel, dim3(unsigned(T + (127 * G + waves - 1) / waves)), dim3(unsigned(64 * waves)), stream,
                         static_cast<const TD*>(dout), static_cast<const TY*>(y), row_of, w, T, int(topk), o, offsets,
                         counts, G, R, dw);
}

hipError_t launch_combine_backward(const void* dout, int dout_bf16, int64_t T, int64_t H, const void* y, int y_bf16,
                                   int64_t R, const int32_t* row_of, const float* w, int64_t topk,
                                   const int32_t* offsets, const int32_t* counts, int64_t G, uint8_t* q, float* s,
                                   float* dw, hipStream_t stream) {
#define FP8FG_CB(D, Y) return run_combine_backward<D, Y>(dout, T, H, y, R, row_of, w, topk, offsets, counts, G, q, s, dw, stream)
    if (dout_bf16) {
        if (y_bf16) FP8FG_CB(uint16_t, uint16_t);
        FP8FG_CB(uint16_t, float);
    }
    if (y_bf16) FP8FG_CB(float, uint16_t);
    FP8FG_CB(float, float);
#undef FP8FG_CB
}

}  // namespace fp8fg
