// gfx950 kernels of the sparse attention's first two steps, and their C entry
// points: the bounds of pages' keys, and the choice of pages by them.  (The
// attention over the chosen pages is in attn.hip.)
#include <algorithm>

#include "kv_device.h"

namespace {

// ------------------------------------------------------------------ codes of 8 bits
// The exponent e of the least 127 * 2^e that holds a finite bf16 number's
// absolute value, from its bits (127 = 1.984375 * 2^6: seven bits of mantissa
// hold 126 / 128 and no more).  Subnormal numbers read as 2^-127: under the limit.
__device__ __forceinline__ int code_exponent(uint32_t bits) {
    const int e = (int)(bits >> 7) - 127 - 6 + ((bits & 127u) > 126u ? 1 : 0);
    return min(max(e, -SP_EXP), SP_EXP);
}
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// Nearest whole number of x * unit within +-127; NaN is 0.  (unit is a power of
// two: the product is exact, or far below a half.)
__device__ __forceinline__ int code(float x, float unit) {
    const float y = fminf(fmaxf(rintf(x * unit), -127.f), 127.f);
    return x == x ? (int)y : 0;
}
__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)d << 24;
}
// bf16 numbers, two in a register, as 16-bit integers of the same order (and back):
// NaN lies past the infinities, on the side of its sign.
__device__ __forceinline__ s16x2_t ordered(s16x2_t x) { return x ^ ((x >> 15) & (short)0x7FFF); }

// ------------------------------------------------------------------ bounds
struct BoundsArgs {
    Kv kv;
    int8_t* codes;
    uint8_t* exps;
    const int32_t* pages;
    int32_t n_pages;
};

// 16 bytes of a token to a lane, so LPT lanes to a token, four tokens to a lane, and as
// many lanes to a page of one head as it has work for: G pages' heads to a wave.  The
// largest and the least are kept as 16-bit integers of the same order, two to a
// register.  The first exchange between lanes leaves the largest to one half of a
// page's lanes and the least (its complement, so that both are maxima) to the other;
// they join and code one of them each.
// Bound by memory, but for the exchanges in small pages: the pages of 48 sequences of up
// to 16384 tokens (8 kv heads, e4m3, pages of 64, 167 MB) take 32 us, 5.2 TB/s, those of
// 16 prompts of up to 2048 (32 heads, bf16, pages of 16, 73 MB, part of them in the
// caches) 13.1 us, 5.5 TB/s; 32000 tokens of 16 heads, e4m3 in pages of 16, of 128
// elements 17.5 us, of 64 10.8.  (With a wave to a page whatever its size, all lanes
// joining both through LDS: 39 and 13.1, 39.5 and 40.4.)  Of that form: two or eight
// loads of a lane under way instead of four 41 and 38 us for the first.  Heads of 64 in
// e4m3 stay at 3.5 to 4 TB/s: the vector units are busy 81% of the time (61% with heads of
// 128), since a page of a head has half the bytes and as many joins and exponents; the
// requests to the cache are as many for each byte.
// From kBoundsPast bytes of keys on, loads go past the caches, which they would only
// fill (a write of so many keys, and of as many values, has left none of them there).
// us without and with that, 16 heads, the same keys again and again, which the caches
// hold as far as they can, and three sets of keys in turn:
//   bf16, 128, pages of 64   132 MB 22/22 26/23   167 27/28 34/29   305 48/50 59/51   508  96/83   96/85
//         64           16    138    21/24 28/25   175 27/33 37/32   319 63/61 65/58   531 109/101 108/96
//   e4m3, 128          64    135    26/26 30/27   171 32/34 38/34   312 66/63 65/58   519 113/104 105/95
//         64           16    148    34/40 36/37   188 43/51 44/45   342 85/87 76/77   571 136/138 125/127: never
constexpr int64_t kBoundsPast = 160000000;
template <int D, bool E4M3, int G, bool PAST>
struct PageBounds {
    static constexpr int LPT = D * (E4M3 ? 1 : 2) / 16, LANES = 64 / G, TOKENS = LANES / LPT;
    static constexpr int N = E4M3 ? 8 : 4, E = 2 * N;  // registers and elements of a lane
    static constexpr int AHEAD = 4;  // loads of a lane that are under way
    static_assert(TOKENS * AHEAD >= 16, "");

    // the lane has the least, not the largest; and it is the one of several that writes
    __device__ __forceinline__ static bool least() { return (threadIdx.x & (G == 1 ? 32 : G == 2 ? 16 : 4)) != 0; }
    __device__ __forceinline__ static bool first() { return (int)(threadIdx.x & (G == 1 ? 31 : G == 2 ? 15 : 11)) < LPT; }

    __device__ __forceinline__ static void values(const char* from, uint32_t scale, u32x4_t (&x)[N / 4]) {
        const u32x4_t* at = reinterpret_cast<const u32x4_t*>(from);
        const u32x4_t raw = PAST ? __builtin_nontemporal_load(at) : *at;
        if constexpr (E4M3) {
            x[0] = dequant8(u32x2_t{raw[0], raw[1]}, scale_of(scale));
            x[1] = dequant8(u32x2_t{raw[2], raw[3]}, scale_of(scale));
        } else {
            x[0] = raw;
        }
    }
    template <typename F>
    __device__ __forceinline__ static void each_token(const Kv& c, int32_t page, int32_t head, F use) {
        const int lane = threadIdx.x % LANES, n = 1 << c.page_shift;
        const char* base = c.k + (E4M3 ? 1 : 2) * kv_off(c, page, head, 0) + 16 * (lane % LPT);
        const uint8_t* scales = c.k_scale + (E4M3 ? scale_off(c, page, head, 0) : 0);
        const int64_t step = (E4M3 ? 1 : 2) * c.token_stride;
        for (int t = AHEAD * (lane / LPT); t < n; t += AHEAD * TOKENS) {  // n is a multiple of AHEAD
            u32x4_t x[AHEAD][N / 4];
            uint32_t exps = 0;
            if constexpr (E4M3) __builtin_memcpy(&exps, scales + t, AHEAD);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) values(base + (t + i) * step, exps >> 8 * i & 255, x[i]);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) use(x[i]);
        }
    }
    __device__ __forceinline__ static s16x2_t joined(s16x2_t x, s16x2_t y) { return __builtin_elementwise_max(x, y); }
    // x and y of this half of the lanes and the other (of 32, or of each 32), or the
    // lower half's x and the upper half's y of both
    template <int HALF>
    __device__ __forceinline__ static s16x2_t across(s16x2_t x, s16x2_t y) {
        const uint32_t a = __builtin_bit_cast(uint32_t, x), b = __builtin_bit_cast(uint32_t, y);
        const auto r = HALF == 32 ? __builtin_amdgcn_permlane32_swap(a, b, false, false)
                                  : __builtin_amdgcn_permlane16_swap(a, b, false, false);
        return joined(__builtin_bit_cast(s16x2_t, (uint32_t)r[0]), __builtin_bit_cast(s16x2_t, (uint32_t)r[1]));
    }
    template <int BY>  // lanes of each 16
    __device__ __forceinline__ static s16x2_t around(s16x2_t x) {
        return joined(x, __builtin_bit_cast(s16x2_t, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x120 + BY, 0xF,
                                                                               0xF, false)));
    }
    __device__ __forceinline__ static s16x2_t in_row(s16x2_t x) {
        if constexpr (LPT <= 4) x = around<4>(x);
        if constexpr (LPT <= 8) x = around<8>(x);
        return x;
    }
    // The largest or the least, two bf16 to a register, and their largest absolute value as bits.
    __device__ __forceinline__ static uint32_t find(const Kv& c, int32_t page, int32_t head, uint32_t (&out)[N]) {
        s16x2_t hi[N], lo[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            hi[j] = s16x2_t{-32768, -32768};
            lo[j] = s16x2_t{32767, 32767};
        }
        each_token(c, page, head, [&](const u32x4_t(&x)[N / 4]) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const s16x2_t y = ordered(__builtin_bit_cast(s16x2_t, (uint32_t)x[j / 4][j % 4]));
                hi[j] = joined(hi[j], y);
                lo[j] = __builtin_elementwise_min(lo[j], y);
            }
        });
        s16x2_t most = {0, 0};
#pragma unroll
        for (int j = 0; j < N; ++j) {
            s16x2_t x;
            if constexpr (G == 1) {
                x = across<32>(hi[j], ~lo[j]);
                x = in_row(across<16>(x, x));
            } else if constexpr (G == 2) {
                x = in_row(across<16>(hi[j], ~lo[j]));
            } else {
                const s16x2_t y = in_row(hi[j]), z = in_row(~lo[j]);
                x = least() ? z : y;
            }
            x = ordered(least() ? ~x : x);
            out[j] = __builtin_bit_cast(uint32_t, x);
            most = joined(most, x & (short)0x7FFF);
        }
        // (a row holds the largest or the least of all elements, or both)
        most = around<1>(around<2>(around<4>(around<8>(most))));
        if constexpr (G == 2) most = across<16>(most, most);
        if constexpr (G == 1) most = across<32>(most, most);
        return (uint32_t)max((int)most[0], (int)most[1]);
    }
};

// Pages with infinities or NaN: the largest and smallest of what is not NaN, and
// the largest finite absolute value, element by element.
template <typename P>
__device__ __forceinline__ uint32_t careful_bounds(const Kv& c, int32_t page, int32_t head, uint32_t (&out)[P::N]) {
    constexpr int E = P::E;
    float hi[E], lo[E];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
        hi[j] = -INFINITY;
        lo[j] = INFINITY;
    }
    P::each_token(c, page, head, [&](const u32x4_t(&x)[P::N / 4]) {
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const uint32_t w = x[j / 8][j % 8 / 2], bits = j & 1 ? w >> 16 : w & 0xFFFFu;
            const float v = __uint_as_float(bits << 16);
            hi[j] = v > hi[j] ? v : hi[j];
            lo[j] = v < lo[j] ? v : lo[j];
            if ((bits & 0x7FFFu) < 0x7F80u) top = max(top, bits & 0x7FFFu);
        }
    });
#pragma unroll
    for (int j = 0; j < E; ++j) {
#pragma unroll
        for (int o = P::LPT; o < P::LANES; o <<= 1) {
            hi[j] = fmaxf(hi[j], __shfl_xor(hi[j], o));
            lo[j] = fminf(lo[j], __shfl_xor(lo[j], o));
        }
        if (hi[j] < lo[j]) hi[j] = lo[j] = 0.f;  // nothing but NaN
    }
#pragma unroll
    for (int j = 0; j < E; j += 2)
        out[j / 2] = __float_as_uint(P::least() ? lo[j] : hi[j]) >> 16 |
                     (__float_as_uint(P::least() ? lo[j + 1] : hi[j + 1]) & 0xFFFF0000u);
    for (int o = 1; o < P::LANES; o <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    return top;
}

template <int D, bool E4M3, int G, bool PAST>
__global__ __launch_bounds__(256) void kv_bounds_kernel(BoundsArgs a) {
    typedef PageBounds<D, E4M3, G, PAST> P;
    const uint32_t units = (uint32_t)a.n_pages * (uint32_t)a.kv.n_kv_heads;
    const uint32_t u = (blockIdx.x * 4 + (G > 1 ? threadIdx.x >> 6 : (uint32_t)wave_id())) * G + (threadIdx.x & 63) / P::LANES;
    if (u - (threadIdx.x & 63) / P::LANES >= units) return;  // (the last wave's other pages: of the last one again)
    const uint32_t unit_of = min(u, units - 1);
    const int32_t page = clamp_page(a.kv, a.pages[unit_of / (uint32_t)a.kv.n_kv_heads]);
    const int32_t head = (int32_t)(unit_of % (uint32_t)a.kv.n_kv_heads);
    uint32_t x[P::N];
    uint32_t top = P::find(a.kv, page, head, x);
    if (__ballot(top >= 0x7F80u)) top = careful_bounds<P>(a.kv, page, head, x);
    const int e = code_exponent(top);
    const float unit = power(-e);
    const int64_t at = (int64_t)page * a.kv.n_kv_heads + head;
    if (P::first()) {
        uint32_t w[P::N / 2];
#pragma unroll
        for (int j = 0; j < P::N; j += 2)
            w[j / 2] = pack4(code(bf16_lo(x[j]), unit), code(bf16_hi(x[j]), unit), code(bf16_lo(x[j + 1]), unit),
                             code(bf16_hi(x[j + 1]), unit));
        int8_t* to = a.codes + (2 * at + P::least()) * D + P::E * (threadIdx.x % P::LPT);
        if constexpr (E4M3) *reinterpret_cast<u32x4_t*>(to) = u32x4_t{w[0], w[1], w[2], w[3]};
        else *reinterpret_cast<u32x2_t*>(to) = u32x2_t{w[0], w[1]};
    }
    if (threadIdx.x % P::LANES == 0) a.exps[at] = (uint8_t)(e + 127);
}

// ------------------------------------------------------------------ select
struct SelectArgs {
    const int8_t* codes;
    const uint8_t* exps;
    const uint16_t* q;
    const lora_sparse_item_t* items;
    const int32_t* table;
    int32_t* selected;
    uint32_t* keys;  // of one launch's items, where they do not fit LDS: [item][head][max_scored]
    int64_t ldq;
    int32_t n_pages, page_shift, n_kv_heads, group, pad_shift;  // 2^pad_shift rows to a token
    int32_t n_seq, n_rows, ld_table, select, first, last, max_scored, item_tokens;
};
struct SelectItem : lora_sparse_item_t {
    const int32_t* table;
    // pages scored of token i (0: it sees them all)
    __device__ __forceinline__ int own(const SelectArgs& a, int i) const { return (pos + i) >> a.page_shift; }
    __device__ __forceinline__ int scored(const SelectArgs& a, int i) const {
        return pos + i < 0 || own(a, i) + 1 <= a.select ? 0 : own(a, i) + 1 - a.last - a.first;
    }
    // there is something to choose
    __device__ __forceinline__ bool scores(const SelectArgs& a) const {
        return a.select > a.first + a.last && scored(a, n - 1) > 0;
    }
};
// Items that do not lie inside the batch are skipped.
__device__ __forceinline__ bool load_select(const SelectArgs& a, int i, SelectItem& it) {
    static_cast<lora_sparse_item_t&>(it) = a.items[i];
    if (it.seq < 0 || it.seq >= a.n_seq || it.row < 0 || it.n < 1 || it.n > a.item_tokens || it.row + (int64_t)it.n > a.n_rows)
        return false;
    it.table = a.table + (int64_t)it.seq * a.ld_table;
    return it.pos + it.n - 1 < 0 || (it.own(a, it.n - 1) < a.ld_table && it.scored(a, it.n - 1) <= a.max_scored);
}

// f over lanes by moves between them: the result of all lanes up to each, within 16
// lanes (row_scan) or the wave; `none` changes nothing.
template <typename F>
__device__ __forceinline__ int row_scan(int x, int none, F f) {
#define SP_STEP(ctrl, rows) x = f(x, __builtin_amdgcn_update_dpp(none, x, ctrl, rows, 0xF, false))
    SP_STEP(0x111, 0xF);  // from 1, 2, 4 and 8 lanes before
    SP_STEP(0x112, 0xF);
    SP_STEP(0x114, 0xF);
    SP_STEP(0x118, 0xF);
    return x;
}
template <typename F>
__device__ __forceinline__ int wave_scan(int x, int none, F f) {
    x = row_scan(x, none, f);
    SP_STEP(0x142, 0xA);  // the last of 16 to the next 16, the last of 32 to the other 32
    SP_STEP(0x143, 0xC);
#undef SP_STEP
    return x;
}
__device__ __forceinline__ int larger(int u, int v) { return (int)max((uint32_t)u, (uint32_t)v); }
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_readlane(wave_scan((int)x, 0, larger), 63);
}

// Scores are the products of a tile of 16 rows (query heads of one or more
// tokens) with 16 pages on the 8-bit matrix unit: sum max(r hi, r lo) =
// max(r, 0) . hi + min(r, 0) . lo.  As whole numbers they are exact; times their
// power of two they are below 2^121 and at least 2^-100, exact in fp32 as well.
//
// Tiles of rows and of pages lie in LDS alike: 2 D bytes a row, max(r, 0) or hi
// first.  A lane's operands: 16 bytes of row lane % 16 for each 64 elements.
template <int D>
struct Operand {
    s32x4_t up[D / 64], down[D / 64];
    __device__ __forceinline__ void read(const char* lds) {
        const int col = threadIdx.x & 15, g = threadIdx.x >> 4 & 3;
#pragma unroll
        for (int s = 0; s < D / 64; ++s) {
            up[s] = *reinterpret_cast<const s32x4_t*>(lds + col * (2 * D) + 16 * k_chunk<D>(col, 4 * s + g));
            down[s] = *reinterpret_cast<const s32x4_t*>(lds + col * (2 * D) + 16 * k_chunk<D>(col, D / 16 + 4 * s + g));
        }
    }
};
template <int D>
__device__ __forceinline__ s32x4_t score(const Operand<D>& rows, const Operand<D>& pages) {
    s32x4_t x = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < D / 64; ++s) {
        x = __builtin_amdgcn_mfma_i32_16x16x64_i8(rows.up[s], pages.up[s], x, 0, 0, 0);
        x = __builtin_amdgcn_mfma_i32_16x16x64_i8(rows.down[s], pages.down[s], x, 0, 0, 0);
    }
    return x;
}

// The item's queries as codes, R tiles of rows, made by all WAVES of a workgroup
// together: D/2 lanes to a row, two elements each.  (Every wave for itself, lane by
// lane as the operand wants them, took longer than the scores of 500 pages.)
// Where a token has more heads than a tile, tiles of heads follow one another:
// code() is called for each, all of them after load().
template <int D, int R, int WAVES>
struct Rows {
    static constexpr int LANES = D / 2, STEP = WAVES * 64 / LANES, N = (16 * R + STEP - 1) / STEP;
    uint32_t x[N];

    __device__ __forceinline__ static int heads(const SelectArgs& a) { return (a.group + 15) >> 4; }
    __device__ __forceinline__ static int row(int j) { return j * STEP + (int)threadIdx.x / LANES; }
    __device__ __forceinline__ static int token(const SelectArgs& a, const SelectItem& it, int r) {
        return min(r >> a.pad_shift, it.n - 1);  // rows of tokens that are not there: of the last one again
    }
    __device__ __forceinline__ void load(const SelectArgs& a, const SelectItem& it, int head, int tile) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int r = row(j);  // (the last head again changes no maximum)
            const int h = min(16 * tile + (r & ((1 << a.pad_shift) - 1)), a.group - 1);
            const int64_t at = (it.row + token(a, it, r)) * a.ldq + ((int64_t)head * a.group + h) * D;
            x[j] = *reinterpret_cast<const uint32_t*>(a.q + at + 2 * (threadIdx.x % LANES));
        }
    }
    // top[token]: the bits of the token's largest finite |q|; starts at zero
    __device__ __forceinline__ void find_top(const SelectArgs& a, const SelectItem& it, uint32_t* top) const {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint32_t lo = x[j] & 0x7FFFu, hi = x[j] >> 16 & 0x7FFFu;
            const int m = row_scan((int)max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u), 0, larger);
            if ((threadIdx.x & 15) == 15) atomicMax(&top[token(a, it, row(j))], (uint32_t)m);
        }
    }
    __device__ __forceinline__ void store(const SelectArgs& a, const SelectItem& it, const uint32_t* top, char* lds) const {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int r = row(j), col = threadIdx.x % LANES;
            if (r >= 16 * R) break;
            const float unit = power(-code_exponent(top[token(a, it, r)]));
            const int c0 = code(bf16_lo(x[j]), unit), c1 = code(bf16_hi(x[j]), unit);
            char* to = lds + r * (2 * D) + 2 * (col % 8);
            const auto put = [&](int c, int u, int v) {
                *reinterpret_cast<uint16_t*>(to + 16 * k_chunk<D>(r & 15, c)) = (uint16_t)((u & 255) | (v & 255) << 8);
            };
            put(col / 8, max(c0, 0), max(c1, 0));
            put(D / 16 + col / 8, min(c0, 0), min(c1, 0));
        }
    }
};

// The bounds of 16 pages, which go through LDS: lanes on end load a page's 2 D bytes
// (as operands, 16 bytes of each of 16 pages to lanes on end, the loads took four
// times as long: the cache serves 64 bytes at a time), and each gets what the
// product wants of page lane % 16 back.
template <int D>
struct Pages16 {
    static constexpr int S = D / 64, CPR = D / 8, RPI = 64 / CPR, LOADS = 16 / RPI;
    u32x4_t raw[LOADS];
    uint32_t exp;         // of page lane % 16
    int32_t ids[LOADS];   // pages that the lane loads of, and page lane % 16: of the tile to load next
    int32_t id;

    __device__ __forceinline__ void look_up(const int32_t* table, int tile, int count) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int j = 0; j < LOADS; ++j) ids[j] = table[(uint32_t)min(16 * tile + RPI * j + lane / CPR, count - 1)];
        id = table[(uint32_t)min(16 * tile + (lane & 15), count - 1)];
    }
    __device__ __forceinline__ void load(const SelectArgs& a, int head) {
        const int8_t* codes = a.codes + (int64_t)head * (2 * D) + 16 * ((threadIdx.x & 63) % CPR);
        const uint32_t page_bytes = (uint32_t)a.n_kv_heads * (2 * D), last = (uint32_t)(a.n_pages - 1);
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
            raw[j] = *reinterpret_cast<const u32x4_t*>(codes + (uint64_t)min((uint32_t)ids[j], last) * page_bytes);
        exp = a.exps[head + (uint64_t)min((uint32_t)id, last) * (uint32_t)a.n_kv_heads];
    }
    __device__ __forceinline__ void store(char* lds) const {
        const int lane = threadIdx.x & 63, col = lane % CPR;
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            const int r = RPI * j + lane / CPR;
            *reinterpret_cast<u32x4_t*>(lds + r * (2 * D) + 16 * k_chunk<D>(r, col)) = raw[j];
        }
    }
};
// An unsigned number of the order of x.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}

// What a workgroup that scores needs of LDS.
template <int D, int R, int WAVES>
struct ScoreLds {
    __align__(16) char pages[WAVES][32 * D];
    __align__(16) char rows[R * 32 * D];
    uint32_t top[16 * R];
};
// Keys of the item's scored pages, a tile of 16 pages to a wave of each of `parts`
// workgroups in turn, for up to R tiles of rows at once.  put(token, page, key,
// again) takes a token's key of one head, or the largest of several, `again` where
// an earlier tile of heads has given some; the same lane takes a page's every time.
template <int D, int R, int WAVES, typename Put>
__device__ __forceinline__ void score_pages(const SelectArgs& a, const SelectItem& it, int head, int part, int parts,
                                            ScoreLds<D, R, WAVES>& lds, Put put) {
    const int w = wave_id(), count = it.scored(a, it.n - 1), end = (count + 15) >> 4, tile = part * WAVES + w, step = parts * WAVES;
    const int rows = R == 1 ? 1 : ((it.n << a.pad_shift) + 15) >> 4;
    const int32_t* table = it.table + a.first;
    Rows<D, R, WAVES> q;
    Pages16<D> p;
    const int heads = q.heads(a);
    p.look_up(table, tile, count);
    q.load(a, it, head, heads - 1);
    for (int i = threadIdx.x; i < 16 * R; i += 64 * WAVES) lds.top[i] = 0;
    __syncthreads();
    for (int t = heads - 1; t > 0; --t) {
        q.find_top(a, it, lds.top);
        q.load(a, it, head, t - 1);
    }
    p.load(a, head);
    p.look_up(table, tile + step, count);
    q.find_top(a, it, lds.top);
    __syncthreads();
    for (int t = 0; t < heads; ++t) {
        if (t > 0) {
            __syncthreads();
            q.load(a, it, head, t);
            p.look_up(table, tile, count);
            p.load(a, head);
            p.look_up(table, tile + step, count);
        }
        q.store(a, it, lds.top, lds.rows);
        __syncthreads();
        Operand<D> r;
        if (R == 1) r.read(lds.rows);
        for (int i = tile; i < end; i += step) {
            wave_sync();
            p.store(lds.pages[w]);
            wave_sync();
            const float unit = scale_of(p.exp);
            if (i + step < end) {
                p.load(a, head);
                p.look_up(table, i + 2 * step, count);
            }
            Operand<D> b;
            b.read(lds.pages[w]);
            const int at = 16 * i + (int)(threadIdx.x & 15), g = threadIdx.x >> 4 & 3;
            for (int x = 0; x < rows; ++x) {
                if (R > 1) r.read(lds.rows + x * 32 * D);
                const s32x4_t y = score<D>(r, b);  // rows 4 g + 0..3 of page lane % 16
                if (at >= count) continue;
                const auto give = [&](int row, int best) {
                    put(min((16 * x + row) >> a.pad_shift, it.n - 1), at, key_of((float)best * unit), t > 0);
                };
                if (R > 1 && a.pad_shift == 0) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) give(4 * g + k, y[k]);
                } else if (R > 1 && a.pad_shift == 1) {
                    give(4 * g, max(y[0], y[1]));
                    give(4 * g + 2, max(y[2], y[3]));
                } else {
                    give(4 * g, max(max(y[0], y[1]), max(y[2], y[3])));
                }
            }
        }
    }
}

template <int WAVES>
struct SelectScratch {
    __align__(16) uint32_t hist[256];
    uint32_t gt[WAVES], eq[WAVES];
};
template <int TEAM>
__device__ __forceinline__ void team_sync() {
    if constexpr (TEAM > 1) __syncthreads();
    else wave_sync();
}

// Writes the page ids of the k largest of n keys, the earlier among equals, in
// order.  A team of waves (the first ones of a workgroup, the others are gone, or one)
// finds the k-th key digit by digit from the first bit in which the keys differ, by
// counting.  A wave goes through a part of the keys of its own, up to 64 HELD of
// them in registers (HELD 0: any number, from where they are each time).
template <int TEAM, int HELD, typename Keys, typename Scratch>
__device__ __forceinline__ void take_largest(const Keys& key, int n, int k, const int32_t* pages, int32_t* out,
                                             Scratch& s) {
    const int lane = threadIdx.x & 63, wave = TEAM > 1 ? wave_id() : 0;
    const int part = (n + 64 * TEAM - 1) / (64 * TEAM) * 64;
    const int begin = min(n, wave * part), end = min(n, begin + part);
    uint32_t held[HELD > 0 ? HELD : 1];
    int32_t ids[HELD > 0 ? HELD : 1];
    if constexpr (HELD > 0) {
#pragma unroll
        for (int j = 0; j < HELD; ++j) ids[j] = pages[min(begin + 64 * j + lane, n - 1)];
#pragma unroll
        for (int j = 0; j < HELD; ++j) held[j] = key(min(begin + 64 * j + lane, n - 1));
    }
    // each(key, there, page id): 64 pages at a time, in order
    const auto all = [&](auto each) {
        if constexpr (HELD > 0) {
#pragma unroll
            for (int j = 0; j < HELD; ++j) {
                if (begin + 64 * j >= end) break;
                each(held[j], begin + 64 * j + lane < end, [&] { return ids[j]; });
            }
        } else {
            for (int i = begin + lane; i < end + lane; i += 64) each(key(min(i, n - 1)), i < end, [&] { return pages[i]; });
        }
    };
    uint32_t most = 0, rest = 0;
    all([&](uint32_t x, bool there, auto) {
        most = max(most, there ? x : 0u);
        rest = max(rest, there ? ~x : 0u);
    });
    most = wave_max(most);
    rest = wave_max(rest);
    if constexpr (TEAM > 1) {
        if (lane == 0) {
            s.gt[wave] = most;
            s.eq[wave] = rest;
        }
        __syncthreads();
        for (int w = 0; w < TEAM; ++w) {
            most = max(most, s.gt[w]);
            rest = max(rest, s.eq[w]);
        }
    }
    const uint32_t least = ~rest;
    // the keys that are taken for certain are above (prefix under mask), `want` of those equal to it
    uint32_t mask = 0xFFFFFFFFu, prefix = most;
    int want = k;
    if (most != least) {
        const int bits = 32 - __clz(most ^ least);
        int shift = max(0, bits - 8);
        mask = bits == 32 ? 0u : 0xFFFFFFFFu << bits;
        prefix &= mask;
        while (true) {
            team_sync<TEAM>();
            if (TEAM == 1 || wave == 0) *reinterpret_cast<u32x4_t*>(s.hist + 4 * lane) = u32x4_t{0, 0, 0, 0};
            team_sync<TEAM>();
            all([&](uint32_t x, bool there, auto) {
                if (there && (x & mask) == prefix) atomicAdd(&s.hist[x >> shift & 255u], 1u);
            });
            team_sync<TEAM>();
            // digits from the largest down, four to a lane
            const u32x4_t c = *reinterpret_cast<const u32x4_t*>(s.hist + 252 - 4 * lane);
            const int sum = (int)(c[0] + c[1] + c[2] + c[3]);
            const int upto = wave_scan(sum, 0, [](int u, int v) { return u + v; });
            const int at = __ffsll((unsigned long long)__ballot(upto >= want)) - 1;
            int above = upto - sum, digit = 255 - 4 * lane, count = (int)c[3];
#pragma unroll
            for (int j = 2; j >= 0; --j)
                if (above + count < want) {
                    above += count;
                    count = (int)c[j];
                    --digit;
                }
            above = __builtin_amdgcn_readlane(above, at);
            digit = __builtin_amdgcn_readlane(digit, at);
            count = __builtin_amdgcn_readlane(count, at);
            want -= above;
            mask |= 255u << shift;
            prefix |= (uint32_t)digit << shift;
            if (count == want || shift == 0) break;
            shift = max(0, shift - 8);
        }
    }
    int taken = 0, equal = 0;
    if constexpr (TEAM > 1) {
        uint32_t gt = 0, eq = 0;
        all([&](uint32_t x, bool there, auto) {
            gt += __popcll(__ballot(there && (x & mask) > prefix));
            eq += __popcll(__ballot(there && (x & mask) == prefix));
        });
        __syncthreads();
        if (lane == 0) {
            s.gt[wave] = gt;
            s.eq[wave] = eq;
        }
        __syncthreads();
        for (int w = 0; w < wave; ++w) {
            taken += s.gt[w];
            equal += s.eq[w];
        }
        taken += min(equal, want);
    }
    const unsigned long long before = (1ull << lane) - 1;
    all([&](uint32_t x, bool there, auto id) {
        const bool same = there && (x & mask) == prefix;
        const unsigned long long eq = __ballot(same);
        const bool take = (there && (x & mask) > prefix) || (same && equal + __popcll(eq & before) < want);
        const unsigned long long now = __ballot(take);
        if (take) out[taken + __popcll(now & before)] = id();
        taken += __popcll(now);
        equal += __popcll(eq);
    });
}

// Token i's row of the result.
template <int TEAM, int HELD, typename Keys, typename Scratch>
__device__ __forceinline__ void select_token(const SelectArgs& a, const SelectItem& it, int head, int i, const Keys& key,
                                             Scratch& s) {
    const int self = TEAM > 1 ? threadIdx.x : threadIdx.x & 63;
    int32_t* out = a.selected + ((int64_t)(it.row + i) * a.n_kv_heads + head) * a.select;
    const int n = it.scored(a, i), own = it.own(a, i);
    if (n == 0) {
        const int all = it.pos + i < 0 ? 0 : own + 1;
        for (int j = self; j < a.select; j += 64 * TEAM) out[j] = j < all ? it.table[j] : -1;
        return;
    }
    for (int j = self; j < a.first + a.last; j += 64 * TEAM) {
        const bool begin = j < a.first;
        out[begin ? j : j + a.select - a.first - a.last] = it.table[begin ? j : own + 1 - a.last + j - a.first];
    }
    const int k = a.select - a.first - a.last;
    if (k == 0) return;
    if (n <= 64 * TEAM * HELD) take_largest<TEAM, HELD>(key, n, k, it.table + a.first, out + a.first, s);
    else take_largest<TEAM, 0>(key, n, k, it.table + a.first, out + a.first, s);
}

// Scores in LDS, and the choice, in one: of a single token (ONE) by 16 waves, the
// first kTeam of which choose, or of several by eight, each of which chooses for tokens of
// its own.  The bounds' bytes are what has to move, but a call ends long before they
// bound it: one token over 500 pages, 8 kv heads, takes 7.5 us, of which 3 are a launch
// and most of the rest the first pass through the code and the chain item, page ids,
// bounds; 32 tokens over up to 2048 pages of 16 16.3 us, 2.4 TB/s; 512 tokens of 32/8
// heads over 500 pages 14.5, 961 of 64/8 over up to 508 32.  (32 tokens with operands
// loaded as the matrix unit wants them, 16 bytes of each page to a lane: 22.7; with codes
// of the queries made by every wave for itself: 18.9.)  Teams of 8 or 16 waves to choose
// are within 5% of four.  Two tiles of a wave under way instead of one: no faster (heads
// of 64), or spilled (128: 19.8 -> 26.7).  Of the 32 us the choice is a quarter.
constexpr int kTeam = 4;
template <int D, int R>
__global__ __launch_bounds__(R == 1 ? 1024 : 64 * SP_WAVES, 4) void select_kernel(SelectArgs a) {
    constexpr bool ONE = R == 1;
    constexpr int WAVES = ONE ? 16 : SP_WAVES;
    extern __shared__ uint32_t keys[];
    __shared__ SelectScratch<kTeam> s[ONE ? 1 : WAVES];
    __shared__ ScoreLds<D, R, WAVES> lds;
    const int head = blockIdx.x % a.n_kv_heads, w = wave_id();
    SelectItem it;
    if (!load_select(a, blockIdx.x / a.n_kv_heads, it)) return;
    if (it.scores(a)) {
        for (int i = threadIdx.x; i < it.n * a.max_scored; i += 64 * WAVES) keys[i] = 0;  // every key is more
        score_pages<D, R, WAVES>(a, it, head, 0, 1, lds, [&](int token, int page, uint32_t x, bool) {
            atomicMax(&keys[token * a.max_scored + page], x);
        });
        __syncthreads();
    }
    if constexpr (ONE) {
        if (w >= kTeam) return;  // a barrier waits for the waves that are left
        select_token<kTeam, 8>(a, it, head, 0, [&](int page) { return keys[page]; }, s[0]);
    } else {
        for (int i = w; i < it.n; i += WAVES)
            select_token<1, 8>(a, it, head, i, [&](int page) { return keys[i * a.max_scored + page]; }, s[w]);
    }
}

// The same for single tokens in two launches, by way of memory.
constexpr int kScoreTiles = 32;  // tiles of 16 pages of a workgroup, about
template <int D>
__global__ __launch_bounds__(256) void score_kernel(SelectArgs a) {
    __shared__ ScoreLds<D, 1, 4> lds;
    const int head = blockIdx.x % a.n_kv_heads;
    SelectItem it;
    if (!load_select(a, blockIdx.x / a.n_kv_heads, it) || !it.scores(a)) return;
    uint32_t* keys = a.keys + (int64_t)blockIdx.x * a.max_scored;
    score_pages<D, 1, 4>(a, it, head, blockIdx.y, gridDim.y, lds, [&](int, int page, uint32_t x, bool again) {
        x = max(x, (uint32_t)__shfl_xor((int)x, 16));
        x = max(x, (uint32_t)__shfl_xor((int)x, 32));
        if ((threadIdx.x & 48) == 0) keys[page] = again ? max(keys[page], x) : x;
    });
}
__global__ __launch_bounds__(1024) void choose_kernel(SelectArgs a) {
    __shared__ SelectScratch<16> s;
    const int head = blockIdx.x % a.n_kv_heads;
    SelectItem it;
    if (!load_select(a, blockIdx.x / a.n_kv_heads, it)) return;
    const uint32_t* keys = a.keys + (int64_t)blockIdx.x * a.max_scored;
    select_token<16, 16>(a, it, head, 0, [&](int page) { return keys[page]; }, s);
}

int32_t check_bounds(const lora_kv_bounds_t* b, const lora_attn_shape_t& s) {
    if (!b || !b->codes || !b->exps || !aligned16(b->codes)) return LORA_EINVAL;
    if (b->n_pages != s.n_pages || b->n_kv_heads != s.n_kv_heads || b->head_dim != s.head_dim) return LORA_ESHAPE;
    return LORA_OK;
}

}  // namespace

extern "C" int32_t lora_sparse_prepare(const lora_attn_shape_t* shape, const lora_sparse_shape_t* sparse, int32_t n_seq,
                                       const int32_t* q_len, const int32_t* kv_len, const int32_t* bounded,
                                       const int32_t* block_table, int64_t ld_table, int32_t* staging,
                                       int64_t staging_capacity, void* dev_staging, void* hip_stream,
                                       lora_sparse_launch_t* out) {
    if (!out) return LORA_EINVAL;
    out->attn.meta = nullptr;  // info may change with an error, and the calls would take it for the old plan's
    if (!dev_staging || !aligned16(dev_staging)) return LORA_EINVAL;
    const int32_t st = lora_sparse_plan(shape, sparse, n_seq, q_len, kv_len, bounded, block_table, ld_table, staging,
                                        staging_capacity, &out->attn.info, &out->info);
    if (st != LORA_OK) return st;
    const hipError_t e = hipMemcpyAsync(dev_staging, staging, (size_t)out->attn.info.n_staged * sizeof(int32_t),
                                        hipMemcpyHostToDevice, reinterpret_cast<hipStream_t>(hip_stream));
    if (e != hipSuccess) return LORA_EHIP;
    out->attn.meta = static_cast<const int32_t*>(dev_staging);
    return LORA_OK;
}

extern "C" int32_t lora_kv_bounds(const lora_sparse_launch_t* L, const lora_kv_t* kv, const lora_kv_bounds_t* bounds,
                                  void* hip_stream) {
    if (!L) return LORA_EINVAL;
    int32_t st = check_kv(&L->attn, kv);
    if (st == LORA_OK) st = check_sparse(*L);
    if (st == LORA_OK) st = check_bounds(bounds, L->attn.info.shape);
    if (st != LORA_OK) return st;
    if (L->info.n_fresh == 0) return LORA_OK;
    BoundsArgs a{to_kv(*kv), bounds->codes, bounds->exps, nullptr, 0};
    typedef void (*fn_t)(BoundsArgs);
    // by the lanes that a page of one head has work for, 16 bytes of four tokens each
#define SP_FORMS(d, e4m3, g) {kv_bounds_kernel<d, e4m3, g, false>, kv_bounds_kernel<d, e4m3, g, true>}
#define SP_NEVER(d, e4m3, g) {kv_bounds_kernel<d, e4m3, g, false>, nullptr}
    static const fn_t fn[2][2][3][2] = {{{SP_FORMS(64, false, 1), SP_FORMS(64, false, 2), {}},
                                         {SP_NEVER(64, true, 1), SP_NEVER(64, true, 2), SP_NEVER(64, true, 4)}},
                                        {{SP_FORMS(128, false, 1), {}, {}},
                                         {SP_FORMS(128, true, 1), SP_FORMS(128, true, 2), {}}}};
#undef SP_FORMS
#undef SP_NEVER
    const bool e4m3 = kv->dtype == LORA_KV_E4M3;
    const int lanes = kv->head_dim * (e4m3 ? 1 : 2) / 16 * kv->page_tokens / 4, form = lanes >= 64 ? 0 : lanes >= 32 ? 1 : 2;
    const int32_t hk = kv->n_kv_heads;
    const bool past = !(e4m3 && kv->head_dim == 64) &&
                      (int64_t)L->info.n_fresh * kv->page_tokens * hk * kv->head_dim * (e4m3 ? 1 : 2) >= kBoundsPast;
    const int32_t most = std::max(1, (int32_t)(kMaxBlocks / hk));  // pages of a launch
    for (int32_t i = 0; i < L->info.n_fresh; i += a.n_pages) {
        a.pages = L->attn.meta + L->info.off_fresh + i;
        a.n_pages = std::min(most, L->info.n_fresh - i);
        const int64_t units = (int64_t)a.n_pages * hk, per = 4 << form;
        if (launch(fn[kv->head_dim == 128][e4m3][form][past], dim3((unsigned)((units + per - 1) / per)), dim3(256),
                   reinterpret_cast<hipStream_t>(hip_stream), a) != hipSuccess)
            return LORA_EHIP;
    }
    return LORA_OK;
}

extern "C" int32_t lora_sparse_select(const lora_sparse_launch_t* L, const lora_kv_bounds_t* bounds, const uint16_t* q,
                                      int64_t ldq, int32_t* selected, float* workspace, int64_t workspace_floats,
                                      void* hip_stream) {
    if (!L) return LORA_EINVAL;
    int32_t st = check_sparse(*L);
    if (st == LORA_OK) st = check_bounds(bounds, L->attn.info.shape);
    if (st != LORA_OK) return st;
    const lora_attn_info_t& I = L->attn.info;
    const lora_sparse_info_t& S = L->info;
    const int32_t d = I.shape.head_dim, hk = I.shape.n_kv_heads;
    if (I.n_rows == 0) return LORA_OK;
    if (bad_rows(q, ldq, (int64_t)I.shape.n_heads * d) || !selected || ((uintptr_t)selected & 3u)) return LORA_EINVAL;
    SelectArgs a;
    memset(&a, 0, sizeof(a));
    a.codes = bounds->codes;
    a.exps = bounds->exps;
    a.q = q;
    a.table = L->attn.meta + I.off_table;
    a.selected = selected;
    a.ldq = ldq;
    a.n_pages = I.shape.n_pages;
    a.page_shift = __builtin_ctz((unsigned)I.shape.page_tokens);
    a.n_kv_heads = hk;
    a.group = I.shape.n_heads / hk;
    while (a.pad_shift < 4 && 1 << a.pad_shift < a.group) ++a.pad_shift;
    a.n_seq = I.n_seq;
    a.n_rows = I.n_rows;
    a.ld_table = I.ld_table;
    a.select = S.shape.select;
    a.first = S.shape.first;
    a.last = S.shape.last;
    a.max_scored = S.max_scored;
    a.item_tokens = S.item_tokens;
    if (a.item_tokens < 1 || a.item_tokens > (16 * SP_ROW_TILES) >> a.pad_shift) return LORA_EINVAL;
    const lora_sparse_item_t* items = reinterpret_cast<const lora_sparse_item_t*>(L->attn.meta + S.off_items);
    const hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
    if (sp_in_lds(S.max_scored, S.item_tokens)) {
        void* p[] = {&a};
        const bool one = S.item_tokens == 1;
        typedef void (*fn_t)(SelectArgs);
        static const fn_t fn[2][3] = {{select_kernel<64, 1>, select_kernel<64, 2>, select_kernel<64, 4>},
                                      {select_kernel<128, 1>, select_kernel<128, 2>, select_kernel<128, 4>}};
        const int form = one ? 0 : S.item_tokens << a.pad_shift <= 32 ? 1 : 2;  // 1, 2 or 4 tiles of rows
        const size_t lds = sizeof(uint32_t) * (size_t)S.max_scored * (size_t)S.item_tokens;
        const int64_t most = std::max<int64_t>(1, kMaxBlocks / 4 / hk);  // items of a launch, of up to 1024 threads
        for (int64_t i = 0; i < S.n_items; i += most) {
            a.items = items + i;
            const dim3 grid((unsigned)(std::min<int64_t>(most, S.n_items - i) * hk));
            if (hipLaunchKernel(reinterpret_cast<const void*>(fn[d == 128][form]), grid, dim3(one ? 1024 : 64 * SP_WAVES), p, lds,
                                stream) != hipSuccess)
                return LORA_EHIP;
        }
        return LORA_OK;
    }
    if (workspace_floats < I.workspace_floats) return LORA_ECAPACITY;
    if (!workspace || !aligned16(workspace)) return LORA_EINVAL;
    if (S.item_tokens != 1) return LORA_EINVAL;
    const int64_t per = (int64_t)S.max_scored * hk, slab = sp_slab(per, S.n_items);
    if (slab * per > I.workspace_floats || slab * hk > kMaxBlocks / 4) return LORA_EINVAL;
    a.keys = reinterpret_cast<uint32_t*>(workspace);
    const int64_t parts = (S.max_scored + 16 * kScoreTiles - 1) / (16 * kScoreTiles);
    for (int64_t i = 0; i < S.n_items; i += slab) {
        a.items = items + i;
        const unsigned blocks = (unsigned)((S.n_items - i < slab ? S.n_items - i : slab) * hk);
        const unsigned gy = (unsigned)std::max<int64_t>(1, std::min(std::min<int64_t>(parts, 4096), kMaxBlocks / blocks));
        if (launch(d == 128 ? score_kernel<128> : score_kernel<64>, dim3(blocks, gy), dim3(256), stream, a) !=
                hipSuccess ||
            launch(choose_kernel, dim3(blocks), dim3(1024), stream, a) != hipSuccess)
            return LORA_EHIP;
    }
    return LORA_OK;
}
