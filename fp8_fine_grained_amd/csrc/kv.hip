// The key/value cache's bookkeeping and its writes (gfx950): a step's pages,
// slots and positions from the requests' lengths, rotary positions, and new keys
// and values quantized into the cache's pages.
#include "elementwise.hpp"
#include "launch.hpp"

namespace fp8fg {

namespace kv_detail {

constexpr int kThreads = 256, kWaves = kThreads / 64;

// Inclusive sums over the wave's lanes, by shifts within the 16-lane rows and
// broadcasts of a row's last lane to the rows behind it
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_dpp(int v) { return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false); }
__device__ __forceinline__ int wave_scan(int v) {
    v = add_dpp<0x111, 0xF>(v);           // row_shr 1, 2, 4, 8
    v = add_dpp<0x112, 0xF>(v);
    v = add_dpp<0x114, 0xF>(v);
    v = add_dpp<0x118, 0xF>(v);
    v = add_dpp<0x142, 0xA>(v);           // row_bcast 15, 31
    return add_dpp<0x143, 0xC>(v);
}
__device__ __forceinline__ int lane63(int v) { return __builtin_amdgcn_readlane(v, 63); }

// Four consecutive values of a lane's requests, 0 past the end
constexpr int kPer = 4, kChunk = 64 * kPer;
__device__ __forceinline__ void load4_until(const int32_t* p, int64_t b, int64_t end, int (&v)[kPer]) {
    if (b + kPer <= end) {
        const int4 w = ld<int4>(p + b);
        v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = b + i < end ? p[b + i] : 0;
    }
}

// The last index i in [0, n) with start[i] <= x (start non-decreasing, start[0] <= x)
__device__ __forceinline__ int last_not_past(const int32_t* start, int n, int32_t x) {
    int lo = 0;
    while (n > 1) {
        const int half = n / 2;
        if (start[lo + half] <= x) lo += half;
        n -= half;
    }
    return lo;
}

// A step's tables.  Request b holds have[b] tokens in ceil(have / page) pages and
// brings add[b] more; the rows of the step are the new tokens in the order of the
// requests.  Every wave forms the sums over all requests, 256 at a time, four to a lane,
// and a workgroup writes the rows and requests that are its own: none waits for another.
// A row that is a page's first token writes the page into the table.  Bound by
// latency: the lengths, a search of eight steps in LDS, the page's number, the stores.
// 256 requests' decode step 4.8 us in a graph (7.2 with 64-bit sums over the
// workgroup, shuffled and joined in LDS), 40 prompts' 37,503 rows 6.6.  Every workgroup walks all lengths: 4096 requests 18, 65,536 195.
struct AssignArgs {
    const int32_t *have, *add, *free_pages, *n_free;
    int64_t B, F, width, T;
    int page_log;
    int32_t *table, *lens, *cu, *positions, *slots, *left;
};
constexpr int kRows = 1024;               // rows of a workgroup
__device__ __forceinline__ int clamp0(int v, int most) { return v < 0 ? 0 : v < most ? v : most; }

__global__ __launch_bounds__(kThreads) void assign(const AssignArgs p) {
    // of each request: its first row, its tokens, the place of its first new page (-1: refused)
    __shared__ __align__(16) int32_t start[kChunk], held[kChunk], first_new[kChunk];
    const int lane = threadIdx.x & 63, T = int(p.T), page = 1 << p.page_log;
    const int row0 = blockIdx.x * kRows, row1 = row0 + kRows < T ? row0 + kRows : T;
    const int n = clamp0(p.n_free[0], int(p.F));
    int rows = 0, used = 0;               // rows and pages so far: T < 2^23, so a chunk's sums fit 32 bits
    int64_t wanted = 0;
    for (int64_t b0 = 0; b0 < p.B; b0 += kChunk) {
        const int64_t b = b0 + lane * kPer;
        int have[kPer], add[kPer], at[kPer], need[kPer], sum = 0;
        load4_until(p.have, b, p.B, have);
        load4_until(p.add, b, p.B, add);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            have[i] = have[i] < 0 ? 0 : have[i];
            add[i] = clamp0(add[i], T);
            sum += add[i];
        }
        const int upto = wave_scan(sum);
        // rows are counted before the pages: a request past the last row brings fewer tokens
        int64_t end = int64_t(rows) + upto - sum;
        sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            at[i] = int(end < T ? end : T);
            end += add[i];
            add[i] = int(end < T ? end : T) - at[i];
            const int64_t pages = (int64_t(have[i]) + page - 1) >> p.page_log;
            need[i] = int(((int64_t(have[i]) + add[i] + page - 1) >> p.page_log) - pages);
            if (pages + need[i] > p.width) need[i] = -1;        // its row of the table does not hold it
            sum += need[i] > 0 ? need[i] : 0;
        }
        const int pages = wave_scan(sum);
        int64_t taken = wanted + pages - sum;
        int32_t first[kPer], lens[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t before = taken;
            taken += need[i] > 0 ? need[i] : 0;
            const bool given = need[i] == 0 || (need[i] > 0 && taken <= n);
            if (given && need[i] > 0) used = int(taken);
            first[i] = !given ? -1 : need[i] > 0 ? int32_t(before) : 0;
            lens[i] = given ? have[i] + add[i] : have[i];
        }
        if (threadIdx.x < 64) {
            st<int4>(start + lane * kPer, int4{at[0], at[1], at[2], at[3]});
            st<int4>(held + lane * kPer, int4{have[0], have[1], have[2], have[3]});
            st<int4>(first_new + lane * kPer, int4{first[0], first[1], first[2], first[3]});
            if ((b0 / kChunk) % gridDim.x == blockIdx.x) {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (b + i < p.B) {
                        p.cu[b + i + 1] = at[i] + add[i];
                        p.lens[b + i] = lens[i];
                    }
            }
        }
        const int chunk0 = rows;
        const int64_t total = int64_t(rows) + lane63(upto);
        rows = int(total < T ? total : T);
        wanted += lane63(pages);
        __syncthreads();
        const int from = row0 > chunk0 ? row0 : chunk0, until = row1 < rows ? row1 : rows;
        const int there = int(p.B - b0 < kChunk ? p.B - b0 : kChunk);
        for (int t = from + int(threadIdx.x); t < until; t += kThreads) {
            const int i = last_not_past(start, there, t);
            const int64_t pos = int64_t(held[i]) + (t - start[i]);
            int64_t slot = -1;
            if (first_new[i] >= 0) {
                const int64_t entry = pos >> p.page_log, k = entry - ((int64_t(held[i]) + page - 1) >> p.page_log);
                int32_t* where = p.table + (b0 + i) * p.width + entry;
                int32_t id;
                if (k >= 0) {
                    id = p.free_pages[n - 1 - first_new[i] - k];
                    if ((pos & (page - 1)) == 0) *where = id;
                } else {
                    id = *where;
                }
                if (id >= 0) slot = (int64_t(id) << p.page_log) + (pos & (page - 1));
                if (slot > 0x7FFFFFFF) slot = -1;
            }
            p.positions[t] = int32_t(pos < 0x7FFFFFFF ? pos : 0x7FFFFFFF);
            p.slots[t] = int32_t(slot);
        }
        if (b0 + kChunk < p.B) __syncthreads();
    }
    for (int t = (row0 > rows ? row0 : rows) + int(threadIdx.x); t < row1; t += kThreads) p.positions[t] = p.slots[t] = -1;
    if (blockIdx.x == 0 && threadIdx.x < 64) {
        // the pages given away: the largest sum that was still covered
        const int top = int(lanes_max<64>(uint32_t(used)));
        if (lane == 0) {
            p.cu[0] = 0;
            p.left[0] = n - top;
            p.left[1] = int32_t(wanted > n ? wanted - n : 0);
        }
    }
}

// The pages of the requests that are done, back on the free list in the order of
// the requests and of their entries, by the same sums.  Bound by latency: 96 of 512 requests, 7000 pages, 6.9 us in a graph,
// of which each chunk of 256 lengths takes two; 4096 requests 19, 65,536 374.
struct ReleaseArgs {
    const int32_t *done, *lens, *table, *n_free;
    int64_t B, F, width;
    int page_log;
    int32_t *free_pages, *lens_out, *left;
};

__global__ __launch_bounds__(kThreads) void release(const ReleaseArgs p) {
    __shared__ __align__(16) int32_t start[kChunk];
    const int lane = threadIdx.x & 63, page = 1 << p.page_log;
    const int64_t row0 = int64_t(blockIdx.x) * kRows, row1 = row0 + kRows;
    const int n = clamp0(p.n_free[0], int(p.F));
    int rows = 0;                         // entries so far, below B * width < 2^31
    for (int64_t b0 = 0; b0 < p.B; b0 += kChunk) {
        const int64_t b = b0 + lane * kPer;
        int done[kPer], len[kPer], count[kPer], sum = 0;
        load4_until(p.done, b, p.B, done);
        load4_until(p.lens, b, p.B, len);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            len[i] = len[i] < 0 ? 0 : len[i];
            const int64_t pages = done[i] ? (int64_t(len[i]) + page - 1) >> p.page_log : 0;
            count[i] = int(pages < p.width ? pages : p.width);
            sum += count[i];
        }
        const int upto = wave_scan(sum);
        if (threadIdx.x < 64) {
            int at = rows + upto - sum;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                start[lane * kPer + i] = at;
                at += count[i];
                if (b + i < p.B && (b0 / kChunk) % gridDim.x == blockIdx.x) p.lens_out[b + i] = done[i] ? 0 : len[i];
            }
        }
        const int chunk0 = rows;
        rows += lane63(upto);
        __syncthreads();
        const int64_t from = row0 > chunk0 ? row0 : chunk0, until = row1 < rows ? row1 : rows;
        const int there = int(p.B - b0 < kChunk ? p.B - b0 : kChunk);
        for (int64_t t = from + threadIdx.x; t < until; t += kThreads) {
            const int i = last_not_past(start, there, int(t));
            if (n + t < p.F) p.free_pages[n + t] = p.table[(b0 + i) * p.width + (t - start[i])];
        }
        if (b0 + kChunk < p.B) __syncthreads();
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.left[0] = int32_t(n + int64_t(rows) < p.F ? n + rows : p.F);
}

// Rotary positions.  A wave takes one token: its lanes form the angles' sines and
// cosines, one pair each, and pass them through LDS; then a lane turns eight
// pairs of one head after another.  Angles are position * frequency in
// revolutions, in 64 bits and what those lose (FP32 would lose them from positions of some
// thousands on, 64 bits alone 2^-21 of a radian at 2^31 radians and more beyond), their fraction, half a turn at the most, its
// sine and cosine in FP32: 2^-23 of each, below the products' own roundings.  Bound by memory: 8192 x 72 heads x 128 in BF16, 302 MB, 59 us, 5.1 TB/s.
struct RopeArgs {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t ldq, ldk, ldqo, ldko, T;
    int Hq, H, D, rot, inverse;            // H: heads of both
    float scale;
    const int32_t* positions;
    const float* freqs;
};
constexpr int kMaxPairs = 128;
// position * freq in revolutions, without the whole ones.  (Contracted, the rounded product would
// be subtracted from without its rounding, which `lost` holds.)
__device__ __forceinline__ float part_of_turn(int32_t position, float freq) {
#pragma clang fp contract(off)
    constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnLost = -0x1.6b01ec5417056p-57;   // 1 / (2 pi)
    const double p = double(position), f = double(freq), angle = p * f, angle_lost = __builtin_fma(p, f, -angle);
    const double turns = angle * kTurn, lost = __builtin_fma(angle, kTurn, -turns) + __builtin_fma(angle, kTurnLost, angle_lost * kTurn);
    const double part = (turns - __builtin_rint(turns)) + lost;     // (lost is below 2^-23, but for angles past 2^31)
    return float(part - __builtin_rint(part));
}

template <class T, bool NEXT>
__global__ __launch_bounds__(kThreads) void rope(const RopeArgs p) {
    __shared__ __align__(16) float cs[kWaves][2][kMaxPairs];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = int64_t(blockIdx.x) * kWaves + wave;
    const int32_t pos = t < p.T ? p.positions[t] : -1;
    const int pairs = p.rot / 2, units = pairs / 8;
    for (int i = lane; i < pairs; i += 64) {
        const float r = part_of_turn(pos, p.freqs[i]);
        float s, c;
        sincospif(2.0f * r, &s, &c);
        cs[wave][0][i] = c * p.scale;
        cs[wave][1][i] = (p.inverse ? -s : s) * p.scale;
    }
    __syncthreads();
    if (pos < 0) return;
    const int per = 64 / units, u = lane % units, first = blockIdx.y * per + lane / units;
    if (lane < per * units) {
        float c[8], s[8];
        load_n<8>(&cs[wave][0][u * 8], c);
        load_n<8>(&cs[wave][1][u * 8], s);
        for (int h = first; h < p.H; h += per * gridDim.y) {
            const T* x = h < p.Hq ? static_cast<const T*>(p.q) + t * p.ldq + h * p.D : static_cast<const T*>(p.k) + t * p.ldk + (h - p.Hq) * p.D;
            T* y = h < p.Hq ? static_cast<T*>(p.q_out) + t * p.ldqo + h * p.D : static_cast<T*>(p.k_out) + t * p.ldko + (h - p.Hq) * p.D;
            float a[8], b[8], ya[8], yb[8];
            if constexpr (NEXT) {
                float w[16], z[16];
                load_n<16>(x + u * 16, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    z[2 * i] = __builtin_fmaf(w[2 * i], c[i], -w[2 * i + 1] * s[i]);
                    z[2 * i + 1] = __builtin_fmaf(w[2 * i + 1], c[i], w[2 * i] * s[i]);
                }
                store_n<16>(y + u * 16, z);
            } else {
                load_n<8>(x + u * 8, a);
                load_n<8>(x + pairs + u * 8, b);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ya[i] = __builtin_fmaf(a[i], c[i], -b[i] * s[i]);
                    yb[i] = __builtin_fmaf(b[i], c[i], a[i] * s[i]);
                }
                store_n<8>(y + u * 8, ya);
                store_n<8>(y + pairs + u * 8, yb);
            }
        }
    }
    // channels that are not turned, where they have to move
    const int rest = (p.D - p.rot) / 8;
    if (rest > 0)
        for (int i = blockIdx.y * 64 + lane; i < rest * p.H; i += 64 * gridDim.y) {
            const int h = i / rest, d = p.rot + (i - h * rest) * 8;
            const T* x = h < p.Hq ? static_cast<const T*>(p.q) + t * p.ldq + h * p.D : static_cast<const T*>(p.k) + t * p.ldk + (h - p.Hq) * p.D;
            T* y = h < p.Hq ? static_cast<T*>(p.q_out) + t * p.ldqo + h * p.D : static_cast<T*>(p.k_out) + t * p.ldko + (h - p.Hq) * p.D;
            if (x != y) {
                Raw<T, 8> w;
                w.load(x + d);
#pragma unroll
                for (int j = 0; j < Raw<T, 8>::W; ++j) st<u32x4>(reinterpret_cast<uint8_t*>(y + d) + 16 * j, w.w[j]);
            }
        }
}

// New keys and values into their pages.  The tokens of a page are a run of
// consecutive rows with consecutive slots, and a wave or a workgroup takes one head's run of keys or
// values.  The scale is the least power of two s with amax <= 448 s (2^-126 at the least), over
// the run and the page's older tokens; when it grows, older codes are re-encoded by the exact factor.  Bound by
// latency (slots, scale, data, maximum, stores in turn): 128 tokens x 8 x 128 in BF16 5.9 us in a graph, 5120
// 13.3 (with four waves a SIMD, which is a round and a quarter of workgroups, 14.8).  Thousands of
// single tokens are bound by the bytes that each writes into its value page's rows, every one a sector of 32: 4096 99 us;
// where no older code moves 86, and 136 MB written for 8.4 MB of codes (pages of 16, whose rows share sectors, 29 and 70).
struct AppendArgs {
    const void *k, *v;
    int64_t ldk, ldv, T, n_slots;
    int H, D, page_log;
    const int32_t* slots;
    uint8_t *kc, *vc;
    float *ks, *vs;
};

// 2^e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), e >= -126; 0 for 0
__device__ __forceinline__ float pow2_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    if (u == 0) return 0.0f;
    int e = int(u >> 23) - 8 + ((u & 0x7FFFFF) > 0x600000);       // biased
    e = e < 1 ? 1 : e;
    return __uint_as_float(uint32_t(e) << 23);
}
// Values to codes' quotients x / s: by the scale's power of two, an exact product, which is all of a scale written here (2^-126
// to 2^120, or 0).  The older tokens' scale of a cache that was filled otherwise may be any other number; what is left of it,
// f in (1, 2), divides by a product with its rounded inverse and one remainder step, which rounds as a division does
// (Markstein's theorem; below 2^-100, where remainders lose bits, the code is 0).  No quotient is above 448, for
// s is no less than pow2_scale's; a subnormal s has values of 0 alone.
struct Exact {
    float r;
    template <int N>
    __device__ __forceinline__ void operator()(float (&v)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= r;
    }
};
struct Divide : Exact {
    float f, rf;
    bool exact;
    __device__ __forceinline__ explicit Divide(float s) {
        const uint32_t two = __float_as_uint(s) & 0x7F800000;
        exact = two == 0 || two == __float_as_uint(s);
        r = __uint_as_float(two == 0 ? 0x3F800000 : two == 0x7F000000 ? 0x00400000 : 0x7F000000 - two);       // 1 / 2^127: subnormal
        f = rf = 1.0f;
        if (!exact) {
            f = s * r;
            rf = 1.0f / f;
        }
    }
    template <int N>
    __device__ __forceinline__ void operator()(float (&v)[N]) const {
        Exact::operator()(v);
        if (!exact) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float q = v[i] * rf;
                v[i] = __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, f, v[i]), rf, q), q);      // (-0 + 0 is 0)
            }
        }
    }
};

__device__ __forceinline__ uint32_t shift_codes(uint32_t w, float f) {
    const v2f lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, 1.0f, false), hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, 1.0f, true);
    return cvt4(lo[0] * f, lo[1] * f, hi[0] * f, hi[1] * f);
}

// Two channels of a row
__device__ __forceinline__ v2f widen2(uint32_t w) { return v2f{__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)}; }
__device__ __forceinline__ v2f widen2(v2f w) { return w; }
template <class T>
struct pair_of {
    typedef v2f type;
};
template <>
struct pair_of<uint16_t> {
    typedef uint32_t type;
};

// A run's place: x its first token's channels, rows `step` elements apart; codes, scale its page's.
// Its team is the wave (team 64) or the workgroup (256), `me` the thread's place in it.
template <class T>
struct Run {
    const T* x;
    int64_t step;
    int count, off, page, D;
    uint8_t* codes;
    float* scale;
    float was;                            // the page's scale so far, 0 for a new page
    int me, team;
    float* part;                          // LDS for the workgroup's waves
};

// The page's scale after a run whose largest magnitude is amax (in any lane), and what
// divides by it; older codes are moved to it, 16 bytes at a time.  VALUES: [channel][token],
// where only the bytes of the older tokens are changed.
template <bool VALUES, class T>
__device__ __forceinline__ Divide new_scale(const Run<T>& r, float amax) {
    float s = fmaxf(r.was, pow2_scale(lanes_max<64>(amax)));
    if (r.team > 64) {                    // (every wave has read the page's scale by now, before one writes it)
        __syncthreads();                  // the last use of part is over
        if ((r.me & 63) == 0) r.part[r.me >> 6] = s;
        __syncthreads();
        s = fmaxf(fmaxf(r.part[0], r.part[1]), fmaxf(r.part[2], r.part[3]));
    }
    if (r.me == 0) *r.scale = s;
    if (r.off > 0 && s > r.was) {
        const float f = r.was / s;
        const int across = VALUES ? (r.off + 15) / 16 : 0, pieces = VALUES ? r.D * across : r.off * r.D / 16;
#pragma unroll 4
        for (int i = r.me; i < pieces; i += r.team) {
            const int row = VALUES ? i / across : 0, at = VALUES ? i - row * across : i;
            uint8_t* c = r.codes + row * r.page + 16 * at;
            u32x4 w = ld<u32x4>(c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t moved = shift_codes(w[j], f);
                const int n = VALUES ? r.off - 16 * at - 4 * j : 4;
                const uint32_t mask = n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : 0xFFFFFFFFu >> (32 - 8 * n);
                w[j] = (moved & mask) | (w[j] & ~mask);
            }
            st<u32x4>(c, w);
        }
        // the new tokens' bytes lie in the same 16-byte pieces of other lanes
        if (VALUES && r.team > 64) __syncthreads();
        else if (VALUES) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    return Divide(s);
}

// A run's data are read once: up to HOLD pieces of a thread stay in registers between
// the maximum and the encoding; longer runs read again.
template <int HOLD, class Load, class Look, class Put, class Scale>
__device__ __forceinline__ void in_two_passes(int pieces, int me, int team, Load load, Look look, Put put, Scale scale) {
    typedef decltype(load(0)) Piece;
    if (pieces <= team * HOLD) {
        Piece w[HOLD];
#pragma unroll
        for (int i = 0; i < HOLD; ++i)
            if (team * i < pieces) w[i] = load(me + team * i < pieces ? me + team * i : pieces - 1);
#pragma unroll
        for (int i = 0; i < HOLD; ++i)
            if (team * i < pieces) look(w[i]);
        const Divide r = scale();
        // (held as they came: the compiler would keep the widened values of the first pass, 119 in place of 91 registers)
#pragma unroll
        for (int i = 0; i < HOLD; ++i)
#pragma unroll
            for (auto& v : w[i].w) asm volatile("" : "+v"(v));
#pragma unroll
        for (int i = 0; i < HOLD; ++i)
            if (me + team * i < pieces) put(me + team * i, w[i], r);
        return;
    }
#pragma unroll 4
    for (int i = me; i < pieces; i += team) look(load(i));
    const Divide r = scale();
    if (!r.exact) {
        for (int i = me; i < pieces; i += team) put(i, load(i), r);
        return;
    }
    // (a branch at each piece would hold up the next ones' loads)
#pragma unroll 4
    for (int i = me; i < pieces; i += team) put(i, load(i), Exact(r));
}

// Keys: eight channels of a token at a time
template <class T>
__device__ __forceinline__ void append_keys(const Run<T>& r) {
    const int per = r.D / 8;
    float amax = 0.0f;
    in_two_passes<sizeof(T) == 2 ? 8 : 4>(
        r.count * per, r.me, r.team,
        [&](int i) {
            Raw<T, 8> w;
            w.load(r.x + int64_t(i / per) * r.step + i % per * 8);
            return w;
        },
        [&](const Raw<T, 8>& w) {
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(w.get(j)));
        },
        [&](int i, const Raw<T, 8>& w, const auto& by_scale) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = w.get(j);
            by_scale(v);
            st<u32x2_t>(r.codes + r.off * r.D + i * 8, u32x2_t{cvt4(v[0], v[1], v[2], v[3]), cvt4(v[4], v[5], v[6], v[7])});
        },
        [&] { return new_scale<false>(r, amax); });
}

// Values, transposed: two channels of a 16-token group of the page at a time, which
// become one 16-byte piece of each channel's row (single bytes where the run does not
// cover the group, whose other tokens read as the run's nearest).
template <class T>
struct Group {
    typename pair_of<T>::type w[16];
};
template <class T>
__device__ __forceinline__ void append_values(const Run<T>& r) {
    const int pairs = r.D / 2, g0 = r.off / 16, groups = (r.off + r.count - 1) / 16 - g0 + 1;
    float amax = 0.0f;
    in_two_passes<sizeof(T) == 2 ? 2 : 1>(
        pairs * groups, r.me, r.team,
        [&](int task) {
            const int g = task / pairs, first = (g0 + g) * 16 - r.off;      // the group's first token, counted from the run's
            Group<T> a;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                int t = first + i;
                t = t < 0 ? 0 : t < r.count ? t : r.count - 1;
                a.w[i] = ld<typename pair_of<T>::type>(r.x + int64_t(t) * r.step + 2 * (task - g * pairs));
            }
            return a;
        },
        [&](const Group<T>& a) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const v2f v = widen2(a.w[i]);
                amax = fmaxf(amax, fmaxf(fabsf(v[0]), fabsf(v[1])));
            }
        },
        [&](int task, const Group<T>& a, const auto& by_scale) {
            const int g = task / pairs, first = (g0 + g) * 16 - r.off;
            uint8_t* c = r.codes + 2 * (task - g * pairs) * r.page + (g0 + g) * 16;
            u32x4 x, y;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const v2f two = widen2(a.w[4 * i + j]);
                    v[j] = two[0];
                    v[4 + j] = two[1];
                }
                by_scale(v);
                x[i] = cvt4(v[0], v[1], v[2], v[3]);
                y[i] = cvt4(v[4], v[5], v[6], v[7]);
            }
            if (first >= 0 && first + 16 <= r.count) {
                st<u32x4>(c, x);
                st<u32x4>(c + r.page, y);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (first + i >= 0 && first + i < r.count) {
                        c[i] = uint8_t(x[i / 4] >> (8 * (i % 4)));
                        c[r.page + i] = uint8_t(y[i / 4] >> (8 * (i % 4)));
                    }
            }
        },
        [&] { return new_scale<true>(r, amax); });
}

// One token, as in a decode step, by a wave: two channels a lane
template <bool VALUES, class T>
__device__ __forceinline__ void append_one(const Run<T>& r) {
    const int lane = threadIdx.x & 63, pairs = r.D / 2;
    typename pair_of<T>::type w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = ld<typename pair_of<T>::type>(r.x + 2 * (lane + 64 * i < pairs ? lane + 64 * i : 0));
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) amax = fmaxf(amax, fmaxf(fabsf(widen2(w[i])[0]), fabsf(widen2(w[i])[1])));
    const Divide by_scale = new_scale<VALUES>(r, amax);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (lane + 64 * i < pairs) {
            float v[2] = {widen2(w[i])[0], widen2(w[i])[1]};
            by_scale(v);
            const uint32_t two = cvt4(v[0], v[1], 0.0f, 0.0f);
            if constexpr (VALUES) {
                uint8_t* c = r.codes + 2 * (lane + 64 * i) * r.page + r.off;
                c[0] = uint8_t(two);
                c[r.page] = uint8_t(two >> 8);
            } else {
                st<uint16_t>(r.codes + r.off * r.D + 2 * (lane + 64 * i), uint16_t(two));
            }
        }
}

// A workgroup looks at `window` (a divisor of 64) rows of one head, its keys or its values, and takes
// the runs that begin in them: three and more a wave each, in turn, fewer the whole
// workgroup one after another.  Bit j of a word says that the j-th row continues the run of the
// row before it.
template <class T>
__global__ __launch_bounds__(kThreads, 5) void append(const AppendArgs p, int window) {
    __shared__ float part[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = blockIdx.y, page = 1 << p.page_log;
    const bool values = blockIdx.z != 0;
    const int64_t row0 = int64_t(blockIdx.x) * window;
    const auto slot_of = [&](int64_t t) { return t >= 0 && t < p.T ? p.slots[t] : -2; };
    const int32_t mine = slot_of(row0 + lane), before = slot_of(row0 + lane - 1), next = slot_of(row0 + 64 + lane), last = slot_of(row0 + 63 + lane);
    const auto continues = [&](int32_t a, int32_t b) { return b >= 0 && int64_t(a) + 1 == b && (b & (page - 1)) != 0; };
    const uint64_t joins = __ballot(continues(before, mine)), joins2 = __ballot(continues(last, next));
    uint64_t heads = __ballot(lane < window && mine >= 0 && mine < p.n_slots) & ~joins;
    const bool together = __popcll(heads) < 3;
    for (int turn = 0; heads; ++turn, heads &= heads - 1) {
        if (!together && turn % kWaves != wave) continue;
        const int first = __builtin_ctzll(heads), slot = __builtin_amdgcn_readlane(mine, first);
        // the run ends before the first row that continues nothing
        uint64_t stop = ~joins & (first < 63 ? ~uint64_t(0) << (first + 1) : 0);
        int end = 64;
        if (stop) {
            end = __builtin_ctzll(stop);
        } else if (joins2 != ~uint64_t(0)) {
            end = 64 + __builtin_ctzll(~joins2);
        } else {
            for (end = 128;; end += 64) {            // a page holds 256 tokens at the most
                stop = ~__ballot(continues(slot_of(row0 + end + lane - 1), slot_of(row0 + end + lane)));
                if (stop) break;
            }
            end += __builtin_ctzll(stop);
        }
        const int64_t t = row0 + first, at = (int64_t(slot) >> p.page_log) * p.H + h, tile = int64_t(page) * p.D;
        Run<T> r;
        r.x = static_cast<const T*>(values ? p.v : p.k) + t * (values ? p.ldv : p.ldk) + h * p.D;
        r.step = values ? p.ldv : p.ldk;
        r.count = end - first;
        r.off = slot & (page - 1);
        r.page = page;
        r.D = p.D;
        r.codes = (values ? p.vc : p.kc) + at * tile;
        r.scale = (values ? p.vs : p.ks) + at;
        r.was = r.off > 0 ? *r.scale : 0.0f;
        r.part = part;
        r.team = together && r.count > 1 ? kThreads : 64;
        r.me = together && r.count > 1 ? threadIdx.x : lane;
        if (r.count == 1) {
            if (together && turn % kWaves != wave) continue;
            if (values) append_one<true>(r);
            else append_one<false>(r);
        } else {
            if (values) append_values(r);
            else append_keys(r);
        }
    }
}

}  // namespace kv_detail

hipError_t launch_kv_assign(const int32_t* have, const int32_t* add, int64_t B, const int32_t* free_pages, const int32_t* n_free,
                            int64_t F, int page_log, int32_t* table, int64_t width, int64_t T, int32_t* lens, int32_t* cu,
                            int32_t* positions, int32_t* slots, int32_t* left, hipStream_t stream) {
    using namespace kv_detail;
    const int64_t blocks = T > 0 ? (T + kRows - 1) / kRows : 1;
    return launch_kernel(assign, dim3(unsigned(blocks)), dim3(kThreads), stream,
                         AssignArgs{have, add, free_pages, n_free, B, F, width, T, page_log, table, lens, cu, positions, slots, left});
}

hipError_t launch_kv_release(const int32_t* done, const int32_t* lens, const int32_t* table, int64_t B, int64_t width, int page_log,
                             int32_t* free_pages, int64_t F, const int32_t* n_free, int32_t* lens_out, int32_t* left,
                             hipStream_t stream) {
    using namespace kv_detail;
    // no more pages than the free list can take come back
    const int64_t most = B * width < F ? B * width : F, blocks = most > 0 ? (most + kRows - 1) / kRows : 1;
    return launch_kernel(release, dim3(unsigned(blocks)), dim3(kThreads), stream,
                         ReleaseArgs{done, lens, table, n_free, B, F, width, page_log, free_pages, lens_out, left});
}

hipError_t launch_rope(const RopeCall& c, hipStream_t stream) {
    using namespace kv_detail;
    const RopeArgs p{c.q, c.k, c.q_out, c.k_out, c.ldq, c.ldk, c.ldqo, c.ldko, c.T, int(c.Hq), int(c.Hq + c.Hkv), int(c.D), int(c.rot),
                     c.inverse, c.scale, c.positions, c.freqs};
    const int units = p.rot / 16, per = 64 / units, passes = (p.H + per - 1) / per;
    // few tokens: their heads over several workgroups, each with the angles again.  us with one / several, 72 heads
    // of 128: 64 tokens of 40 heads 5.4 / 4.4, 1024 10.1 / 8.4, 2048 15.0 / 14.6, 4096 28.0 / 28.2
    const dim3 grid(unsigned((c.T + kWaves - 1) / kWaves), unsigned(c.T <= 2048 ? passes : 1));
    if (c.bf16)
        return launch_kernel(c.interleaved ? rope<uint16_t, true> : rope<uint16_t, false>, grid, dim3(kThreads), stream, p);
    return launch_kernel(c.interleaved ? rope<float, true> : rope<float, false>, grid, dim3(kThreads), stream, p);
}

hipError_t launch_kv_append(const KvAppendCall& c, hipStream_t stream) {
    using namespace kv_detail;
    const AppendArgs p{c.k, c.v, c.ldk, c.ldv, c.T, c.n_pages << c.page_log, int(c.H), int(c.D), c.page_log, c.slots, c.kc, c.vc, c.ks, c.vs};
    // Few rows: each may begin a run of its own; many: most continue one.  About a thousand workgroups: us with windows of
    // 4 / 16 / 64 rows, 8 heads of 128, single tokens: 128 5.9 / 7.5 / 18, 512 12.1 / 11.3 / 20, 2048 46 / 45 / 43 (32 rows: 42);
    // runs: 5120 rows 36 / 22 / 15, 1250 14.0 / 11.1 / 10.1 (32 rows: 9.6)
    int window = 4;
    while (window < 64 && window * 512 < c.T * c.H) window *= 2;
    return launch_kernel(c.bf16 ? append<uint16_t> : append<float>, dim3(unsigned((c.T + window - 1) / window), unsigned(c.H), 2),
                         dim3(kThreads), stream, p, window);
}

}  // namespace fp8fg
