// Attention of new tokens over the 8-bit cache (gfx950).
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale q_i . k_j - m_i)
//
// over the keys j that token i sees, in one pass with a running maximum m.
// Keys and values are E4M3 codes times one scale per page and head.  K's codes
// are widened exactly to BF16 and multiplied with the BF16 queries, V's exactly
// to FP16 and multiplied with FP16 probabilities, sums in FP32.  (The matrix units take 16 bits:
// half a step of FP16 is 2^-11 of a probability, an eighth of the output's own rounding to BF16; as
// BF16 a probability would cost as much as that.)  Units of the sums and lse go through the
// hardware's approximate reciprocal and logarithm, which costs a probability 2^-18 at the most.
//
// A tile is 64 tokens of one head, S^T = K Q^T of it four 16-token products.
// The 16 x 16 result of the matrix instruction leaves row 4 g + i of a 16-lane
// group g in register i, so with row n of product j holding token
// 16 (n / 4) + 4 j + n % 4, group g ends up with tokens 16 g .. 16 g + 15 of one
// query row: exactly the operand P^T of O^T = V^T P^T, in which group g's
// lanes supply 16 consecutive tokens.  No probability moves between lanes, a
// lane's V operand is 16 consecutive bytes of the value page ([channel][token]),
// and its 16 tokens lie in one page, whose scales are two registers.
#include "elementwise.hpp"
#include "launch.hpp"

namespace fp8fg {

namespace attend_detail {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kTile = 64;                 // tokens of a tile
// Tiles that a split holds at the least, and tables that hold no more than kWhole tiles are not
// split: 1024 tokens are four steps of each wave, and joining takes a second launch (four requests of up to 601
// tokens, 32 / 8 heads: 10.4 us whole, 15.9 split)
constexpr int kMinTiles = 8, kWhole = 16;
constexpr int kSlots = 512;               // workgroups that run at a time: two on each of 256 CUs
// Probabilities are held times 2^11, relative to a maximum that is raised only when
// a score passes it by a factor of 2^4: at most 2^15, and FP16 keeps them normal
// down to 2^-25.  (Were every new maximum taken, some row of a tile would have one most of
// the time, and all sums be multiplied.)
constexpr float kPBias = 11.0f, kSlack = 4.0f;
// What waves and parts join is a sum of 2^31 values at the most, each below 2^128 and times a probability held as up to
// 2^15: it is held times 2^-48, so that it stays in FP32's range until the division by the probabilities' sum
constexpr float kDown = 0x1p-48f, kUp = 0x1p48f;

struct Args {
    const uint16_t* q;
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *table, *cu, *lens;
    int64_t ldq, n_pages, width, B, T;
    int Hq, Hkv, G, page_log;             // G: query heads of a key/value head
    float scale2;                         // softmax scale * log2(e)
    uint16_t* out;
    float* lse;
    int32_t* list;                        // workspace: number of items, and from list + 8 on the items; null: not listed
    int32_t* desc;                        // [T][G] x (splits, first part, row of it)
    float* parts;                         // unjoined results: maxima, sums of probabilities, sums of values times kDown
    int64_t most_parts;                   // room for them
    int target;                           // workgroups wanted for each key/value head
};

// What a workgroup does: rows tile * ROWS .. of request b (n tokens from row cu of q on), the
// split-th of `splits` parts of its keys
struct Item {
    int32_t b, cu, n, len, tile, split, splits, part;
};

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

// Four consecutive requests of a lane: their rows and tokens, with what lies outside
// the batch and the tables cut off, row tiles and tiles of keys
constexpr int kPer = 4, kChunk = 64 * kPer;
template <int ROWS>
struct Requests {
    int cu[kPer + 1], n[kPer], len[kPer], tiles[kPer], kt[kPer];
    __device__ __forceinline__ void read(const Args& p, int64_t b0) {
        const int room = int(p.width << p.page_log), lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i <= kPer; ++i) {
            const int64_t b = b0 + lane * kPer + i;
            cu[i] = p.cu[b < p.B ? b : p.B];
            if (i < kPer) len[i] = b < p.B ? p.lens[b] : 0;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int end = cu[i + 1] < p.T ? cu[i + 1] : int(p.T);
            cu[i] = cu[i] < 0 ? 0 : cu[i];
            n[i] = end > cu[i] ? end - cu[i] : 0;
            len[i] = len[i] < 0 ? 0 : len[i] > room ? room : len[i];
            tiles[i] = int((int64_t(n[i]) * p.G + ROWS - 1) / ROWS);
            kt[i] = (len[i] + kTile - 1) / kTile;
        }
    }
    __device__ __forceinline__ float work() const {
        float w = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) w += float(tiles[i]) * float(kt[i]);
        return w;
    }
};

// Tiles of a part, from the work of all requests: so many that about `target` workgroups do
// all of it (no less for the roundings of a sum in FP32)
__device__ __forceinline__ int part_of(const Args& p, float work) {
    const float want = ceilf(work * (1.0f + 0x1p-20f) / float(p.target));
    return !p.parts ? 1 << 30 : want < float(kMinTiles) ? kMinTiles : want > 0x1p30f ? 1 << 30 : int(want);
}
__device__ __forceinline__ int splits_of(int kt, int per) { return kt > per ? (kt + per - 1) / per : 1; }

// The requests' row tiles and their splits, numbered in order: the me-th.  Up to 256
// requests every wave finds it from the lengths, four requests to a lane, without
// LDS or a barrier; more are listed by a launch of their own.
template <int ROWS, bool CLASSES>
__device__ __forceinline__ bool find_item(const Args& p, int me, Item& it) {
    if (p.list) {
        const int32_t* at = p.list + 8 + int64_t(me) * 8;
        const int4 a = ld<int4>(at), b = ld<int4>(at + 4);
        const auto get = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
        it = Item{get(a.x), get(a.y), get(a.z), get(a.w), get(b.x), get(b.y), get(b.z), get(b.w)};
        return me < p.list[0] && it.n > 0;
    }
    const int lane = threadIdx.x & 63;
    Requests<ROWS> r;
    r.read(p, 0);
    const int per = part_of(p, lanes_sum<64>(r.work()));
    // CLASSES: requests whose parts are long come first, in four classes by their share of the
    // longest, so that what starts last is short.  (The list of more than 256 requests goes without.)  Three chunks
    // of up to 2048 tokens on 1024 to 8192: 528 / 461 us without and with.  Parts of a decode step are alike; there the classes' scans cost 0.7 us and save nothing.
    int splits[kPer], size[kPer], longest = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        splits[i] = 1;
        size[i] = r.kt[i];
        if (p.parts) {                    // (a division costs tens of instructions)
            splits[i] = splits_of(r.kt[i], per);
            if (CLASSES) size[i] = splits[i] > 1 ? (r.kt[i] + splits[i] - 1) / splits[i] : r.kt[i];
        }
        longest = size[i] > longest && r.tiles[i] > 0 ? size[i] : longest;
    }
    if (CLASSES) longest = __builtin_amdgcn_readfirstlane(int(lanes_max<64>(uint32_t(longest))));
    int items0 = 0, parts0 = 0;
    for (int cls = CLASSES ? 3 : 0; cls >= 0; --cls) {
        const int over = cls > 0 ? int(int64_t(longest) * cls / 4) : -1, upto = CLASSES && cls < 3 ? int(int64_t(longest) * (cls + 1) / 4) : 0x7FFFFFFF;
        int items = 0, parts = 0, here[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            here[i] = size[i] > over && size[i] <= upto ? r.tiles[i] * splits[i] : 0;
            items += here[i];
            parts += splits[i] > 1 ? here[i] : 0;
        }
        const int i1 = wave_scan(items), p1 = wave_scan(parts);
        int at = me - items0 - (i1 - items);
        const uint64_t who = __ballot(at >= 0 && at < items);
        if (who) {
            int part = parts0 + p1 - parts;
            Item mine{};                  // tile: the item's place among its request's
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (at >= 0 && at < here[i]) mine = Item{lane * kPer + i, r.cu[i], r.n[i], r.len[i], at, 0, splits[i], part};
                at -= here[i];
                part += splits[i] > 1 ? here[i] : 0;
            }
            const int src = __builtin_ctzll(who);
            const auto get = [&](int v) { return __builtin_amdgcn_readlane(v, src); };
            it = Item{get(mine.b), get(mine.cu), get(mine.n), get(mine.len), get(mine.tile), 0, get(mine.splits), get(mine.part)};
            if (it.splits > 1) {
                const int tile = it.tile / it.splits;
                it.split = it.tile - tile * it.splits;
                it.part += tile * it.splits;
                it.tile = tile;
            }
            return it.splits == 1 || (it.part >= 0 && it.part + it.splits <= p.most_parts);
        }
        items0 += lane63(i1);
        parts0 += lane63(p1);
    }
    return false;
}

// The same for more than 256 requests, once for all workgroups: a wave for each 256 of them sums
// the work of all and the items before its own, and writes its own out.  1000 requests of up
// to 500 tokens, 8 heads: 259 us with every wave finding its item among all, 154 with the list; 300 of up to 8192,
// one head: 72 / 74.
template <int ROWS>
__global__ __launch_bounds__(64) void list_items(const Args p, int64_t room) {
    const int lane = threadIdx.x & 63;
    const int64_t own = int64_t(blockIdx.x) * kChunk;
    Requests<ROWS> r;
    float work = 0.0f;
    if (p.parts) {
#pragma unroll 2
        for (int64_t b0 = 0; b0 < p.B; b0 += kChunk) {
            r.read(p, b0);
            work += r.work();
        }
    }
    const int per = part_of(p, lanes_sum<64>(work));
    int items0 = 0, parts0 = 0;
#pragma unroll 2
    for (int64_t b0 = 0; b0 < own; b0 += kChunk) {
        r.read(p, b0);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int splits = splits_of(r.kt[i], per), all = r.tiles[i] * splits;
            items0 += all;
            parts0 += splits > 1 ? all : 0;
        }
    }
    items0 = lane63(wave_scan(items0));
    parts0 = lane63(wave_scan(parts0));
    r.read(p, own);
    int splits[kPer], items = 0, parts = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        splits[i] = splits_of(r.kt[i], per);
        items += r.tiles[i] * splits[i];
        parts += splits[i] > 1 ? r.tiles[i] * splits[i] : 0;
    }
    const int i1 = wave_scan(items), p1 = wave_scan(parts);
    int64_t at = int64_t(items0) + i1 - items;
    int part = parts0 + p1 - parts;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        // (items and parts that no room was counted for, which sound offsets do not have, are left out)
        for (int tile = 0; tile < r.tiles[i] && at >= 0 && at < room; ++tile) {
            const bool fits = splits[i] == 1 || (part >= 0 && part + splits[i] <= p.most_parts);
            for (int split = 0; split < splits[i] && at < room; ++split, ++at) {
                int32_t* to = p.list + 8 + at * 8;
                st<int4>(to, int4{int32_t(own) + lane * kPer + i, r.cu[i], fits ? r.n[i] : 0, r.len[i]});
                st<int4>(to + 4, int4{tile, split, fits ? splits[i] : 1, splits[i] > 1 ? part : 0});
            }
            part += splits[i] > 1 ? splits[i] : 0;
        }
    }
    if (own + kChunk >= p.B && lane == 0) p.list[0] = items0 + lane63(i1);
}

// Token and query head of a row tile's rows: one division for the tile, the rest by a
// reciprocal in FP32 (exact for quotients' operands below 2^21: they are at most G + 128)
struct Rows {
    int token, rest, G;
    float inverse;
    __device__ __forceinline__ Rows(int first, int G_) : token(first / G_), rest(first - token * G_), G(G_), inverse(1.0f / float(G_)) {}
    __device__ __forceinline__ int token_of(int r) const { return token + int((float(rest + r) + 0.5f) * inverse); }
    __device__ __forceinline__ int head_of(int r, int t) const { return rest + r - (t - token) * G; }
};

template <bool HI>
__device__ __forceinline__ uint32_t to_bf16(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(int(w), 1.0f, HI));
}
template <bool HI>
__device__ __forceinline__ uint32_t to_f16(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(w), 1.0f, HI));
}
__device__ __forceinline__ v8bf wide_bf16(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(v8bf, u32x4{to_bf16<false>(a), to_bf16<true>(a), to_bf16<false>(b), to_bf16<true>(b)});
}
__device__ __forceinline__ v8h wide_f16(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(v8h, u32x4{to_f16<false>(a), to_f16<true>(a), to_f16<false>(b), to_f16<true>(b)});
}

// Over the four 16-lane groups: rows are swapped in pairs, then halves
template <class Op>
__device__ __forceinline__ float groups_reduce(float v, Op op) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    const uint32_t a = s[0], b = s[1];
    v = op(__uint_as_float(a), __uint_as_float(b));
    const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    const uint32_t c = t[0], d = t[1];
    return op(__uint_as_float(c), __uint_as_float(d));
}
__device__ __forceinline__ float groups_max(float v) { return groups_reduce(v, MaxOp()); }
__device__ __forceinline__ float groups_sum(float v) { return groups_reduce(v, SumOp()); }

// max over the two halves of the wave
__device__ __forceinline__ float halves_max(float v) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    const uint32_t a = s[0], b = s[1];
    return fmaxf(__uint_as_float(a), __uint_as_float(b));
}

// A row of O is held in units of its own `ref`: the largest value scale of the tile's pages that
// the row sees a token of, while that lies within [ref / 64, ref] the one before, so that the sums
// are seldom multiplied; but no less than 2^-40 of the largest so far (FP32 holds the sums in such units)
// and 2^-100.  (A unit from all of the tile's pages would take the probabilities of a row below
// FP16's range for a page that only later tokens see.)
__device__ __forceinline__ float unit_of(float top, float largest, float ref) {
    const float want = fmaxf(fmaxf(top, largest * 0x1p-40f), 0x1p-100f);
    return want > ref || want < ref * 0x1p-6f ? want : ref;
}
// 1 / unit, to 2^-21 of it: from 2^126 on a subnormal number, which the instruction would flush
__device__ __forceinline__ float per_unit(float unit) { return __builtin_amdgcn_rcpf(unit * 0x1p-8f) * 0x1p-8f; }

// the bytes of w (tokens first .. first + 3) that lie before `end`
__device__ __forceinline__ uint32_t keep_bytes(uint32_t w, int first, int end) {
    const int n = end - first;
    return n >= 4 ? w : n <= 0 ? 0u : w & (0xFFFFFFFFu >> (32 - 8 * n));
}

// 16 NR query rows of one key/value head and a part of their keys.  The four waves
// take every fourth tile; a wave widens a tile's codes once for all its rows.  Bound by the
// stream of codes: 607 MB (64 requests of 1025 to 8193 tokens, 64 / 8 heads, D = 128) in 115 us, 5.2 TB/s, what a copy
// reaches; matrix units busy 0.08, vector instructions 0.35 of the time.
template <int D, int NR, bool ONCE>
__global__ __launch_bounds__(kThreads, 2) void attend(const Args p) {
    constexpr int ROWS = 16 * NR, KC = D / 64, DT = D / 16;
    constexpr bool kAhead = D <= 192;     // registers for it
    __shared__ __align__(16) float joined[kWaves][ROWS * D];
    __shared__ float stat[kWaves][2][ROWS];
    Item it{};
    if (!find_item<ROWS, false>(p, blockIdx.x, it)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4, kvh = blockIdx.y;
    const int before = it.len - it.n;
    const auto sees = [&](int t) { return t < it.n ? (before + t < it.len ? before + t : it.len - 1) : -1; };
    // this lane's query rows, and the last key that each sees
    const Rows rows(it.tile * ROWS, p.G);
    int tq[NR], hq[NR], last[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        tq[r] = rows.token_of(16 * r + col);
        hq[r] = kvh * p.G + rows.head_of(16 * r + col, tq[r]);
        last[r] = sees(tq[r]);
    }
    const int end_tq = rows.token_of(ROWS - 1), least = sees(rows.token), most = sees(end_tq < it.n ? end_tq : it.n - 1);
    const int kt = most < 0 ? 0 : most / kTile + 1;
    const int per = it.splits > 1 ? (kt + it.splits - 1) / it.splits : kt, kt0 = it.split * per, kt1 = kt0 + per < kt ? kt0 + per : kt;
    const int32_t* table = p.table + int64_t(it.b) * p.width;
    const int64_t page_bytes = int64_t(D) << p.page_log;

    v8bf qf[NR][KC][2];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 w{0u, 0u, 0u, 0u};
                if (tq[r] < it.n) w = ld<u32x4>(p.q + int64_t(it.cu + tq[r]) * p.ldq + hq[r] * D + 64 * c + 16 * g + 8 * h);
                qf[r][c][h] = __builtin_bit_cast(v8bf, w);
            }
    v4f o[NR][DT];
    float m[NR], l[NR], ref[NR], largest[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        m[r] = -__builtin_inff();
        l[r] = ref[r] = largest[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < DT; ++i) o[r][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // The pages of a tile's tokens: of the group whose keys this lane loads and of
    // the lane's own group, -1 where there is none
    const int mask = (1 << p.page_log) - 1;
    const auto page_of = [&](int tile, int group) {
        const int token = tile * kTile + 16 * group;
        return token < it.len ? table[token >> p.page_log] : -1;
    };
    const auto exists = [&](int32_t id) { return id >= 0 && id < p.n_pages; };
    // Keys of the next tile are loaded while this one's values are multiplied, values
    // of this tile while its keys are
    int tile = kt0 + wave;
    int32_t kid = -1, vid = -1, kid2 = -1, vid2 = -1;
    u32x4 kraw[4][KC], vraw[DT];
    const auto load_keys = [&](int tile, int32_t id) {
        const uint8_t* kp = p.kc + (int64_t(exists(id) ? id : 0) * p.Hkv + kvh) * page_bytes +
                            ((tile * kTile + 16 * (col >> 2)) & mask) * D + (col & 3) * D + 16 * g;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < KC; ++c) kraw[j][c] = ld<u32x4>(kp + 4 * j * D + 64 * c);
    };
    if (tile < kt1) {
        kid = page_of(tile, col >> 2);
        vid = page_of(tile, g);
        if (tile + kWaves < kt1) {
            kid2 = page_of(tile + kWaves, col >> 2);
            vid2 = page_of(tile + kWaves, g);
        }
        if (kAhead) load_keys(tile, kid);
    }
    for (; tile < kt1; tile += kWaves) {
        const int t0 = tile * kTile;
        const bool good = exists(vid);
        const int64_t at = int64_t(good ? vid : 0) * p.Hkv + kvh;
        const float ksc = good ? p.ks[at] * p.scale2 : 0.0f, vsc = good ? p.vs[at] : 0.0f;
        const uint8_t* vp = p.vc + at * page_bytes + ((t0 + 16 * g) & mask) + (int64_t(col) << p.page_log);
        const auto load_values = [&] {
#pragma unroll
            for (int d = 0; d < DT; ++d) vraw[d] = ONCE ? ld_once<u32x4>(vp + (int64_t(16 * d) << p.page_log)) : ld<u32x4>(vp + (int64_t(16 * d) << p.page_log));
        };
        if (kAhead) load_values();
        else load_keys(tile, kid);
        v4f s[NR][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int r = 0; r < NR; ++r) s[r][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const u32x4 w = kraw[j][c];
                const v8bf a = wide_bf16(w[0], w[1]), b = wide_bf16(w[2], w[3]);
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    s[r][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, qf[r][c][0], s[r][j], 0, 0, 0);
                    s[r][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, qf[r][c][1], s[r][j], 0, 0, 0);
                }
            }
        }
        kid = kid2;
        vid = vid2;
        if (tile + kWaves < kt1) {
            if (kAhead) load_keys(tile + kWaves, kid);
            if (tile + 2 * kWaves < kt1) {
                kid2 = page_of(tile + 2 * kWaves, col >> 2);
                vid2 = page_of(tile + 2 * kWaves, g);
            }
        }
        if (!kAhead) load_values();
        const float all = groups_max(vsc);
        // scores in units of log2; keys out of sight at -inf
        const bool masked = t0 + kTile - 1 > least || !__all(good);
        v8h pf[NR][2];
        float factor[NR];
        bool same = true;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int seen = good ? last[r] - (t0 + 16 * g) : -1;     // the last of the lane's tokens in sight
            float mt = -__builtin_inff();
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[r][j][i] *= ksc;
                    if (masked && 4 * j + i > seen) s[r][j][i] = -__builtin_inff();
                    mt = fmaxf(mt, s[r][j][i]);
                }
            mt = groups_max(mt);
            const float m_new = mt > m[r] + kSlack ? mt : m[r], m_use = m_new == -__builtin_inff() ? 0.0f : m_new;
            const float alpha = __builtin_amdgcn_exp2f(m[r] - m_use);
            m[r] = m_new;
            const float top = masked ? groups_max(seen >= 0 ? vsc : 0.0f) : all;
            largest[r] = fmaxf(largest[r], top);
            const float unit = unit_of(top, largest[r], ref[r]), inverse = per_unit(unit);
            factor[r] = unit == ref[r] ? alpha : alpha * (ref[r] * inverse);
            ref[r] = unit;
            const float ratio = fminf(vsc * inverse, 1.0f);        // (above 1: a page out of sight)
            same = same && factor[r] == 1.0f;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = __builtin_amdgcn_exp2f(s[r][j][i] - (m_use - kPBias));
                    sum += e;
                    pf[r][j >> 1][(j & 1) * 4 + i] = _Float16(e * ratio);
                }
            l[r] = __builtin_fmaf(l[r], alpha, sum);
        }
        if (masked) {                     // codes past the last token are not numbers
            const int end = !good ? 0 : it.len - (t0 + 16 * g);
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) vraw[d][i] = keep_bytes(vraw[d][i], 4 * i, end);
        }
        if (!__all(same)) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int d = 0; d < DT; ++d) o[r][d] *= factor[r];
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const u32x4 w = vraw[d];
            const v8h a = wide_f16(w[0], w[1]), b = wide_f16(w[2], w[3]);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                o[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pf[r][0], o[r][d], 0, 0, 0);
                o[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, pf[r][1], o[r][d], 0, 0, 0);
            }
        }
    }

    // the four waves' results joined
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        l[r] = groups_sum(l[r]);
        if (g == 0) {
            stat[wave][0][16 * r + col] = m[r];
            stat[wave][1][16 * r + col] = l[r];
        }
    }
    __syncthreads();
    const auto joint = [&](int row, float& M, float& L) {
        M = stat[0][0][row];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) M = fmaxf(M, stat[w][0][row]);
        const float use = M == -__builtin_inff() ? 0.0f : M;
        L = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) L = __builtin_fmaf(stat[w][1][row], __builtin_amdgcn_exp2f(stat[w][0][row] - use), L);
    };
    const bool split = it.splits > 1;
    float* part = p.parts + (int64_t(it.part + it.split) * p.Hkv + kvh) * (ROWS * (D + 2));
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int row = 16 * r + col;
        float M, L;
        joint(row, M, L);
        const float mine = __builtin_amdgcn_exp2f(m[r] - (M == -__builtin_inff() ? 0.0f : M)) * kDown;
#pragma unroll
        for (int d = 0; d < DT; ++d)  // [row][channel], the 16-byte pieces of a row swapped by row
            st<v4f>(&joined[wave][row * D + (((4 * d + g) ^ col) * 4)], o[r][d] * mine * ref[r]);
        if (wave == 0 && g == 0) {
            if (split) {
                part[row] = M;
                part[ROWS + row] = L;
                if (p.desc && it.split == 0 && kvh == 0 && tq[r] < it.n)
                    st<int4>(p.desc + 4 * (int64_t(it.cu + tq[r]) * p.G + (hq[r] - kvh * p.G)), int4{it.splits, it.part, row, 0});
            } else if (tq[r] < it.n) {
                if (p.lse)
                    p.lse[int64_t(it.cu + tq[r]) * p.Hq + hq[r]] = L > 0.0f ? (M + __log2f(L) - kPBias) * 0.6931471805599453f : -__builtin_inff();
                if (p.desc && kvh == 0) st<int4>(p.desc + 4 * (int64_t(it.cu + tq[r]) * p.G + (hq[r] - kvh * p.G)), int4{1, 0, 0, 0});
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS * D / 4; i += kThreads) {
        const int r = i / (D / 4), c = i - r * (D / 4);
        const int t = rows.token_of(r);
        if (t >= it.n) continue;
        v4f v = ld<v4f>(&joined[0][r * D + ((c ^ (r & 15)) * 4)]);
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += ld<v4f>(&joined[w][r * D + ((c ^ (r & 15)) * 4)]);
        if (split) {
            st<v4f>(part + 2 * ROWS + r * D + 4 * c, v);
            continue;
        }
        float M, L;
        joint(r, M, L);
        const float inv = L > 0.0f ? 1.0f / L : 0.0f;
        const float out[4] = {v[0] * inv * kUp, v[1] * inv * kUp, v[2] * inv * kUp, v[3] * inv * kUp};
        store_n<4>(p.out + (int64_t(it.cu + t) * p.Hq + kvh * p.G + rows.head_of(r, t)) * D + 4 * c, out);
    }
}

// Many query rows: each of the four waves holds 32 rows, and all of them read a
// tile's keys and values from LDS, where they lie widened (BF16 and FP16), in two
// buffers: while a tile is multiplied the next one's codes are on their way in
// registers.  The products are 32 x 32 x 16, again S^T = K Q^T and O^T = V^T P^T: row n =
// 8 b + 4 h + i of a 32-token product holds token 16 h + 4 b + i, so that lane half h ends up with
// tokens 16 h .. 16 h + 15 of a row, one page's, in order.  16-byte pieces of LDS rows are
// swapped by row, so that eight lanes' pieces meet different banks.  Bound by the vector instructions
// beside the products (9.7 for each): 512 tokens on 30,000, 32 / 8 heads, D = 128, 296 us with the join,
// 0.85 PFLOP/s; three chunks of 512 to 2048 on 1024 to 8192 293 to 512 us, 0.83 to 0.87 PFLOP/s.
typedef float v16f __attribute__((ext_vector_type(16)));

template <int D>
__global__ __launch_bounds__(kThreads, D <= 128 ? 2 : 1) void attend_wide(const Args p) {
    constexpr int ROWS = 32 * kWaves, KC = D / 64, DT = D / 32;
    __shared__ __align__(16) uint16_t keys[2][kTile * D], values[2][kTile * D];
    __shared__ float scales[2][2][4];     // [buffer][keys, values][group of 16 tokens]; values' -1: no page
    Item it{};
    const int kvh = blockIdx.x % p.Hkv;
    if (!find_item<ROWS, true>(p, blockIdx.x / p.Hkv, it)) return;
    it.tile = int((int64_t(it.n) * p.G + ROWS - 1) / ROWS) - 1 - it.tile;       // the last rows see the most keys: they start first
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 31, h = lane >> 5, quad = threadIdx.x & 3;
    const int before = it.len - it.n;
    const auto sees = [&](int t) { return t < it.n ? (before + t < it.len ? before + t : it.len - 1) : -1; };
    const Rows rows(it.tile * ROWS, p.G);
    const int tq = rows.token_of(32 * wave + col), hq = kvh * p.G + rows.head_of(32 * wave + col, tq), last = sees(tq);
    const bool live = tq < it.n;
    const int end_tq = rows.token_of(ROWS - 1);
    const int least = sees(rows.token_of(32 * wave)), most = sees(end_tq < it.n ? end_tq : it.n - 1);
    const int kt = most < 0 ? 0 : most / kTile + 1;
    const int per = it.splits > 1 ? (kt + it.splits - 1) / it.splits : kt, kt0 = it.split * per, kt1 = kt0 + per < kt ? kt0 + per : kt;
    const int32_t* table = p.table + int64_t(it.b) * p.width;
    const int mask = (1 << p.page_log) - 1;

    v8bf qf[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        u32x4 w{0u, 0u, 0u, 0u};
        if (live) w = ld<u32x4>(p.q + int64_t(it.cu + tq) * p.ldq + hq * D + 16 * c + 8 * h);
        qf[c] = __builtin_bit_cast(v8bf, w);
    }
    v16f o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f, ref = 0.0f, largest = 0.0f;

    // The page of group `quad` of a tile.  A wave brings the keys of group `wave`; values
    // come by quads of lanes, four groups of a channel side by side.
    // (What is loaded here is looked at only when it is used: a comparison would wait for it.)
    const auto page_of = [&](int tile) {
        const uint32_t token = uint32_t(tile) * kTile + 16 * quad;          // (two tiles past the end, near 2^31)
        return token < uint32_t(it.len) ? table[token >> p.page_log] : -1;
    };
    const uint32_t n_pages = uint32_t(p.n_pages), tile_bytes = uint32_t(D) << p.page_log;       // n_pages * Hkv < 2^30
    const auto exists = [&](int32_t id) { return uint32_t(id) < n_pages; };
    const uint32_t value_row = threadIdx.x / 4;
    u32x4 kraw[KC], vraw[KC];
    float kscale, vscale;
    const auto fetch = [&](int tile, int32_t id) {
        const int32_t kid = __builtin_amdgcn_readlane(id, wave);
        const uint32_t k_at = (exists(kid) ? kid : 0) * uint32_t(p.Hkv) + kvh, at = (exists(id) ? id : 0) * uint32_t(p.Hkv) + kvh;
        const uint8_t* kp = p.kc + uint64_t(k_at) * tile_bytes + uint32_t(((tile * kTile + 16 * wave) & mask) * D);
        const uint8_t* vp = p.vc + (uint64_t(at) * tile_bytes + (uint32_t((tile * kTile + 16 * quad) & mask) + (value_row << p.page_log)));
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            kraw[i] = ld<u32x4>(kp + uint32_t((lane + 64 * i) * 16));
            vraw[i] = ld<u32x4>(vp + (uint32_t(64 * i) << p.page_log));
        }
        kscale = p.ks[at];
        vscale = p.vs[at];
    };
    // Places of 16-byte pieces: rows of 16 pieces (or a multiple) start in the same bank,
    // rows of 8 (or an odd multiple) in two
    const auto key_at = [&](int n, int c) { return n * D + ((c ^ (D % 128 == 0 ? n & 15 : (n >> 1) & 7)) * 8); };
    const auto value_at = [&](int d, int c) { return d * kTile + ((c ^ ((d >> 1) & 7)) * 8); };
    // the fetched tile's values without what is past the last token: those codes are not numbers
    const auto cut = [&](int tile, int32_t id) {
        const bool there = exists(id);
        if ((tile + 1) * kTile > it.len || !__all(there)) {
            const int end = !there ? 0 : it.len - (tile * kTile + 16 * quad);
#pragma unroll
            for (int i = 0; i < KC; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) vraw[i][j] = keep_bytes(vraw[i][j], 4 * j, end);
        }
    };
    // the fetched tile, widened, into buffer `to`
    const auto put = [&](int32_t id, int to) {
        const bool there = exists(id);
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            const int at = lane + 64 * i, r = at / (D / 16), c = 2 * (at % (D / 16));
            // token 16 wave + r: row n of the 32-token product wave / 2
            const int n = 32 * (wave >> 1) + 8 * (r >> 2) + 4 * (wave & 1) + (r & 3);
            const u32x4 w = kraw[i];
            st<v8bf>(&keys[to][key_at(n, c)], wide_bf16(w[0], w[1]));
            st<v8bf>(&keys[to][key_at(n, c + 1)], wide_bf16(w[2], w[3]));
            const u32x4 v = vraw[i];
            const int d = threadIdx.x / 4 + 64 * i;
            st<v8h>(reinterpret_cast<v8h*>(&values[to][value_at(d, 2 * quad)]), wide_f16(v[0], v[1]));
            st<v8h>(reinterpret_cast<v8h*>(&values[to][value_at(d, 2 * quad + 1)]), wide_f16(v[2], v[3]));
        }
        if (threadIdx.x < 4) {
            // never 0: a masked score times it stays -inf (2^-149 times any other one is 0 to the exponential)
            scales[to][0][quad] = there ? fmaxf(kscale * p.scale2, 0x1p-149f) : 0x1p-149f;
            scales[to][1][quad] = there ? vscale : -1.0f;
        }
    };
    int32_t id = page_of(kt0), id2 = page_of(kt0 + 1);
    if (kt0 < kt1) {
        fetch(kt0, id);
        cut(kt0, id);
        put(id, 0);
    }
    __syncthreads();
    for (int tile = kt0; tile < kt1; ++tile) {
        const int buf = (tile - kt0) & 1, t0 = tile * kTile;
        id = id2;
        id2 = page_of(tile + 2);
        if (tile + 1 < kt1) fetch(tile + 1, id);
        v16f s[2];
        float ksc[2], vsc[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            ksc[t] = scales[buf][0][2 * t + h];
            vsc[t] = scales[buf][1][2 * t + h];
#pragma unroll
            for (int i = 0; i < 16; ++i) s[t][i] = 0.0f;
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
            for (int t = 0; t < 2; ++t)
                s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ld<v8bf>(&keys[buf][key_at(32 * t + col, 2 * c + h)]), qf[c], s[t], 0, 0, 0);
        // six keys' pieces ahead of the products: 425 -> 418 us for three chunks of up to 2048 tokens
        __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
        for (int c = 0; c < D / 8 - 6; ++c) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, 6, 0);
        float vis = fmaxf(vsc[0], vsc[1]);            // of the pages in sight
        if (t0 + kTile - 1 > least || !__all(vsc[0] >= 0.0f && vsc[1] >= 0.0f)) {
            vis = 0.0f;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int seen = vsc[t] >= 0.0f ? last - (t0 + 32 * t + 16 * h) : -1;
                vis = seen >= 0 ? fmaxf(vis, vsc[t]) : vis;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i > seen) s[t][i] = -__builtin_inff();
            }
        }
        float mt = -__builtin_inff();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float top = s[t][0];
#pragma unroll
            for (int i = 1; i < 16; ++i) top = fmaxf(top, s[t][i]);
            mt = fmaxf(mt, top * ksc[t]);
        }
        mt = halves_max(mt);
        const float m_new = mt > m + kSlack ? mt : m, m_use = m_new == -__builtin_inff() ? 0.0f : m_new;
        const float alpha = __builtin_amdgcn_exp2f(m - m_use);
        m = m_new;
        const float top = halves_max(vis);
        largest = fmaxf(largest, top);
        const float unit = unit_of(top, largest, ref);
        const float inverse = per_unit(unit), factor = unit == ref ? alpha : alpha * (ref * inverse);
        ref = unit;
        if (!__all(factor == 1.0f)) {
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= factor;
        }
        if (tile + 1 < kt1) cut(tile + 1, id);
        // Probabilities are formed times their page's value scale over `ref`, as a term of the
        // exponent (below 2^-60 FP16 has nothing left of them, above 1 the page is out of sight), and
        // summed without it.  The second half's run beside the first half's products, and beside its own products the next
        // tile is widened (what is put past the end is not used).
        v8h pf[2][2];
        l *= alpha;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float ratio = __builtin_amdgcn_fmed3f(vsc[t] * inverse, 0x1p-60f, 1.0f);
            const float bias = kPBias - m_use + __builtin_amdgcn_logf(ratio);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], ksc[t], bias));
                sum += e;
                pf[t][i >> 3][i & 7] = _Float16(e);
            }
            l = __builtin_fmaf(sum, __builtin_amdgcn_rcpf(ratio), l);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const v8h v = ld<v8h>(&values[buf][value_at(32 * d + col, 4 * t + 2 * h + k)]);
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, pf[t][k], o[d], 0, 0, 0);
                }
        put(id, buf ^ 1);
        __syncthreads();
    }

    l += __shfl_xor(l, 32, 64);
    if (!live) return;
    const bool split = it.splits > 1;
    const int r = 32 * wave + col;
    const int64_t at = int64_t(it.cu + tq) * p.Hq + hq;
    if (split) {
        float* part = p.parts + (int64_t(it.part + it.split) * p.Hkv + kvh) * (ROWS * (D + 2));
        if (h == 0) {
            part[r] = m;
            part[ROWS + r] = l;
        }
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int b = 0; b < 4; ++b)
                st<v4f>(part + 2 * ROWS + r * D + 32 * d + 8 * b + 4 * h,
                        v4f{o[d][4 * b], o[d][4 * b + 1], o[d][4 * b + 2], o[d][4 * b + 3]} * kDown * ref);
    } else {
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const float out[4] = {o[d][4 * b] * inv * ref, o[d][4 * b + 1] * inv * ref, o[d][4 * b + 2] * inv * ref,
                                      o[d][4 * b + 3] * inv * ref};
                store_n<4>(p.out + at * D + 32 * d + 8 * b + 4 * h, out);
            }
        if (h == 0 && p.lse) p.lse[at] = l > 0.0f ? (m + __log2f(l) - kPBias) * 0.6931471805599453f : -__builtin_inff();
    }
    if (p.desc && it.split == 0 && kvh == 0 && h == 0)
        st<int4>(p.desc + 4 * (int64_t(it.cu + tq) * p.G + (hq - kvh * p.G)), int4{it.splits, it.part, r, 0});
}

// The splits of a query row joined, a workgroup for each: D / 4 threads of four
// channels side by side, 1024 / D splits at a time, each with a running maximum of its
// own; they meet in LDS in a fixed order.  Bound by latency: 5.1 us for 64 requests of 64 heads, four to ten parts each.
template <int D, int ROWS>
__global__ __launch_bounds__(kThreads) void join(const Args p) {
    constexpr int PER = D / 4, SIDE = kThreads / PER;
    __shared__ __align__(16) float sums[SIDE][D];
    __shared__ float tops[SIDE], totals[SIDE];
    const int64_t row = blockIdx.x;
    const int kvh = blockIdx.y, used = p.cu[p.B];
    const int4 d = ld<int4>(p.desc + 4 * row);
    const int splits = d.x, first = d.y, r = d.z;
    if (row >= int64_t(used) * p.G || splits <= 1 || first < 0 || splits > p.most_parts - first || r < 0 || r >= ROWS) return;
    const float* part = p.parts + (int64_t(first) * p.Hkv + kvh) * (ROWS * (D + 2)) + r;
    const int64_t step = int64_t(p.Hkv) * (ROWS * (D + 2));
    const int side = threadIdx.x / PER, c = threadIdx.x % PER;
    float M = -__builtin_inff(), L = 0.0f;
    v4f v{0.0f, 0.0f, 0.0f, 0.0f};
    if (side < SIDE) {
#pragma unroll 4
        for (int s = side; s < splits; s += SIDE) {
            const float m = part[s * step], l = part[s * step + ROWS];
            const v4f o = ld<v4f>(part - r + s * step + 2 * ROWS + r * D + 4 * c);
            const float top = fmaxf(M, m), use = top == -__builtin_inff() ? 0.0f : top;
            const float f = __builtin_amdgcn_exp2f(M - use), h = __builtin_amdgcn_exp2f(m - use);
            M = top;
            L = L * f + l * h;
            v = v * f + o * h;
        }
        st<v4f>(&sums[side][4 * c], v);
        if (c == 0) {
            tops[side] = M;
            totals[side] = L;
        }
    }
    __syncthreads();
    if (side != 0) return;
#pragma unroll
    for (int i = 1; i < SIDE; ++i) M = fmaxf(M, tops[i]);
    const float use = M == -__builtin_inff() ? 0.0f : M, f0 = __builtin_amdgcn_exp2f(tops[0] - use);
    L *= f0;
    v *= f0;
#pragma unroll
    for (int i = 1; i < SIDE; ++i) {
        const float f = __builtin_amdgcn_exp2f(tops[i] - use);
        L = __builtin_fmaf(totals[i], f, L);
        v += ld<v4f>(&sums[i][4 * c]) * f;
    }
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
    const int64_t t = row / p.G, at = t * p.Hq + kvh * p.G + (row - t * p.G);
    const float out[4] = {v[0] * inv * kUp, v[1] * inv * kUp, v[2] * inv * kUp, v[3] * inv * kUp};
    store_n<4>(p.out + at * D + 4 * c, out);
    if (c == 0 && p.lse) p.lse[at] = L > 0.0f ? (M + __log2f(L) - kPBias) * 0.6931471805599453f : -__builtin_inff();
}

// The same for many rows of few splits: D / 4 threads a row, which take its splits one after
// another, 1024 / D rows a workgroup (chunk of 2048 tokens on 2000, 16 / 4 heads: the whole call 94 us with a workgroup for each row,
// 83 so)
template <int D, int ROWS, bool HEADS>
__global__ __launch_bounds__(kThreads) void join_rows(const Args p) {
    constexpr int PER = D / 4, SIDE = kThreads / PER;
    const int side = threadIdx.x / PER, c = threadIdx.x % PER, used = p.cu[p.B];
    const int64_t row = int64_t(blockIdx.x) * SIDE + side;
    if (side >= SIDE || row >= p.T * p.G || row >= int64_t(used) * p.G) return;
    const int4 d = ld<int4>(p.desc + 4 * row);
    const int splits = d.x, first = d.y, r = d.z;
    if (splits <= 1 || first < 0 || splits > p.most_parts - first || r < 0 || r >= ROWS) return;
    const int64_t step = int64_t(p.Hkv) * (ROWS * (D + 2)), t = row / p.G;
    for (int kvh = HEADS ? 0 : blockIdx.y; kvh < p.Hkv; ++kvh) {
        const float* part = p.parts + (int64_t(first) * p.Hkv + kvh) * (ROWS * (D + 2)) + r;
        float M = -__builtin_inff(), L = 0.0f;
        v4f v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
            const float m = part[s * step], l = part[s * step + ROWS];
            const v4f o = ld<v4f>(part - r + s * step + 2 * ROWS + r * D + 4 * c);
            const float top = fmaxf(M, m), use = top == -__builtin_inff() ? 0.0f : top;
            const float f = __builtin_amdgcn_exp2f(M - use), h = __builtin_amdgcn_exp2f(m - use);
            M = top;
            L = L * f + l * h;
            v = v * f + o * h;
        }
        const float inv = L > 0.0f ? 1.0f / L : 0.0f;
        const int64_t at = t * p.Hq + kvh * p.G + (row - t * p.G);
        const float out[4] = {v[0] * inv * kUp, v[1] * inv * kUp, v[2] * inv * kUp, v[3] * inv * kUp};
        store_n<4>(p.out + at * D + 4 * c, out);
        if (c == 0 && p.lse) p.lse[at] = L > 0.0f ? (M + __log2f(L) - kPBias) * 0.6931471805599453f : -__builtin_inff();
        if (!HEADS) break;
    }
}

constexpr int kWideRows = 32 * kWaves;
struct Plan {
    int64_t tiles, items, parts;          // bounds: row tiles, workgroups, unjoined results, per key/value head
    int target;
    int64_t list, desc, parts_at, bytes;  // places in the workspace, and its size
};
inline Plan plan_of(const AttendCall& c, int rows) {
    Plan r;
    const int64_t G = c.Hq / c.Hkv, seqs = c.B < c.T ? c.B : c.T, kt = ((c.width << c.page_log) + kTile - 1) / kTile;
    r.tiles = c.T * G / rows + seqs;
    // Parts of equal length, about as many as fill whole rounds of workgroups: every row
    // tile adds half a part, its last one.  us with 512 / 768 / 1024 / 2048 parts: one
    // request of 32,768 tokens, 8 heads, 22 / 27 / 27 / 28; two of 131,072, 4 heads, 44 / 56 / 52 / 69;
    // 64 of 1024 to 8192, 8 heads, 132 / 119 / 126 / 139
    const int64_t all = (c.T * G / rows > seqs ? c.T * G / rows : seqs) * c.Hkv;
    const int64_t rounds = (3 * all / 2 + kSlots - 1) / kSlots;
    r.target = int(((rounds > 1 ? rounds : 1) * kSlots - all / 2 + c.Hkv - 1) / c.Hkv);
    // no part needs to be shorter than half of what one place does in all (and the workspace stays small)
    if (r.target > (2 * kSlots + c.Hkv - 1) / c.Hkv) r.target = int((2 * kSlots + c.Hkv - 1) / c.Hkv);
    // Many rows are split only where their tiles do not fill the chip: chunks of 1024 and 256
    // tokens on 16,000 and 2000, 421 us whole, 210 split; one of 2048 on 2000 109 / 84; six of up to 500 on up
    // to 2000 79 / 85; three of up to 2048 on up to 8192, 960 tiles, 413 / 437.  Where they do, and each of several requests
    // brings many, only tiles longer than a place's share are, which the host cannot see: 2048 and 512 tokens on up to
    // 16,384 494 / 409, five of 512 to 2048 on 1024 to 8192, where none is, 579 / 582 for the empty second launch.
    // (A single token on a very long context is then one workgroup's: 131,072 tokens beside that chunk take 3.6 ms.)
    if (rows == kWideRows && all > kSlots) r.target = seqs > 1 && c.T * G > 512 * seqs ? int((kSlots + c.Hkv - 1) / c.Hkv) : 1;
    const bool split = kt > kWhole && r.target > 1;
    // a tile has one item more than the work's share at the most, a split one twice as many
    // (the work is summed in FP32), and no more than its keys' whole splits
    const int64_t share = r.target + 1, most = split ? r.tiles * ((kt + kMinTiles - 1) / kMinTiles - 1) : 0;
    r.items = r.tiles + (share < most ? share : most);
    r.parts = split ? 2 * int64_t(r.target) + 2 : 0;
    r.list = 0;
    r.desc = c.B > kChunk ? 32 + r.items * 32 : 0;
    r.parts_at = r.desc + (split ? c.T * G * 16 : 0);
    r.bytes = r.parts_at + r.parts * c.Hkv * rows * (c.D + 2) * 4;
    return r;
}

// Rows of a workgroup, by what the requests bring on average: sixteen, thirty-two, or four waves' 32
// over one copy in LDS.  (The host knows no more.  Where a few chunks lift the average, single tokens beside them take
// the wide kernel too: 63 of them on 1024 to 8192 tokens, 116 us alone, with a chunk of 2048 tokens on 4096, 364 alone, 563
// in one call, 64 / 8 heads.)  us, on caches of up to 3000 tokens: 64 requests of 8 heads and D = 128 with 16 rows each, 16 and 32
// a workgroup 56 / 62, with 24 rows 85 / 65; with 40, 50 and 60 rows, 32 and 128 a workgroup 92 / 92, 103 / 93, 116 / 95,
// with 80 144 / 98; 60 rows of four requests 21 / 26, of 32 requests of two heads at D = 256 48 / 46.
inline int rows_of(const AttendCall& c) {
    const int64_t seqs = c.B < c.T ? c.B : c.T, rows = c.T * (c.Hq / c.Hkv);
    return rows > 64 * seqs || (rows > 48 * seqs && seqs * c.Hkv >= kSlots) ? kWideRows : c.D <= 128 && rows > 16 * seqs ? 32 : 16;
}

template <int D, int NR>
hipError_t run(const AttendCall& c, const Args& p, const Plan& plan, hipStream_t stream) {
    // Values that no other workgroup reads pass the caches by.  Without and with, us: 64 requests of 1025 to 8193
    // tokens, 8 heads, 128 / 118 (D = 128), 73 / 69 (64); with 24 to 48 rows each, 49 / 51, 50 / 49, 93 / 96
    auto kernel = attend<D, NR, false>;
    if constexpr (NR == 1) {
        if (c.T * p.G <= 16 * (c.B < c.T ? c.B : c.T)) kernel = attend<D, NR, true>;
    }
    if (const hipError_t e = launch_kernel(kernel, dim3(unsigned(plan.items), unsigned(c.Hkv)), dim3(kThreads), stream, p)) return e;
    if (plan.parts == 0) return hipSuccess;
    return launch_kernel(join<D, 16 * NR>, dim3(unsigned(c.T * p.G), unsigned(c.Hkv)), dim3(kThreads), stream, p);
}

template <int D>
hipError_t run_wide(const AttendCall& c, const Args& p, const Plan& plan, hipStream_t stream) {
    // a head's workgroups side by side: with eight heads each XCD reads one head's keys and values
    if (const hipError_t e = launch_kernel(attend_wide<D>, dim3(unsigned(plan.items * c.Hkv)), dim3(kThreads), stream, p)) return e;
    if (plan.parts == 0) return hipSuccess;
    constexpr int SIDE = 4 * kThreads / D;
    // (where most rows have nothing to join, one workgroup sees to all heads: 3 us in place of 6 for nothing)
    const bool few = c.T * p.G / kWideRows * c.Hkv > kSlots;
    return launch_kernel(few ? join_rows<D, kWideRows, true> : join_rows<D, kWideRows, false>, dim3(unsigned((c.T * p.G + SIDE - 1) / SIDE), few ? 1 : unsigned(c.Hkv)),
                         dim3(kThreads), stream, p);
}

template <int D>
hipError_t run_any(const AttendCall& c, const Args& p, const Plan& plan, int rows, hipStream_t stream) {
    if (rows == kWideRows) return run_wide<D>(c, p, plan, stream);
    if constexpr (D <= 128) {
        if (rows == 32) return run<D, 2>(c, p, plan, stream);
    }
    return run<D, 1>(c, p, plan, stream);
}

}  // namespace attend_detail

int64_t attend_workspace(const AttendCall& c) { return attend_detail::plan_of(c, attend_detail::rows_of(c)).bytes; }

hipError_t launch_attend(const AttendCall& c, hipStream_t stream) {
    using namespace attend_detail;
    const int rows = rows_of(c);
    const Plan plan = plan_of(c, rows);
    // both launches' grids, before the first
    if (!grid_fits(rows == kWideRows ? plan.items * c.Hkv : plan.items, kThreads) ||
        (plan.parts && !grid_fits(c.T * (c.Hq / c.Hkv), kThreads)))
        return hipErrorInvalidConfiguration;
    Args p{c.q, c.kc, c.vc, c.ks, c.vs, c.table, c.cu, c.lens, c.ldq, c.n_pages, c.width, c.B, c.T, int(c.Hq), int(c.Hkv), int(c.Hq / c.Hkv),
           c.page_log, c.scale * 1.4426950408889634f, c.out, c.lse, nullptr, nullptr, nullptr, plan.parts, plan.target};
    uint8_t* w = static_cast<uint8_t*>(c.workspace);
    if (plan.parts) {
        p.desc = reinterpret_cast<int32_t*>(w + plan.desc);
        p.parts = reinterpret_cast<float*>(w + plan.parts_at);
    }
    if (c.B > kChunk) {
        p.list = reinterpret_cast<int32_t*>(w + plan.list);
        const auto kernel = rows == 16 ? list_items<16> : rows == 32 ? list_items<32> : list_items<kWideRows>;
        if (const hipError_t e = launch_kernel(kernel, dim3(unsigned((c.B + kChunk - 1) / kChunk)), dim3(64), stream, p, plan.items)) return e;
    }
    switch (c.D) {
        case 64: return run_any<64>(c, p, plan, rows, stream);
        case 128: return run_any<128>(c, p, plan, rows, stream);
        case 192: return run_any<192>(c, p, plan, rows, stream);
        default: return run_any<256>(c, p, plan, rows, stream);
    }
}

}  // namespace fp8fg
