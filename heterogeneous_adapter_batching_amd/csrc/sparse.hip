// gfx950 kernels of the sparse attention's first two steps, and their C entry
// points: the bounds of pages' keys, and the choice of pages by them.  (The
// attention over the chosen pages is lora_attn's kernel, in attn.hip.)
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

// A wave takes a page of one head: 16 bytes of a token to a lane, so LPT lanes to
// a token and 64 / LPT tokens at once, joined over the lanes at the end.  Largest
// and smallest are kept as ordered 16-bit integers, two to a register.
template <int D, bool E4M3>
struct PageBounds {
    static constexpr int LPT = D * (E4M3 ? 1 : 2) / 16, TOKENS = 64 / LPT, N = E4M3 ? 8 : 4;  // registers of elements
    static constexpr int AHEAD = 4;  // loads of a lane that are under way
    s16x2_t hi[N], lo[N];

    __device__ __forceinline__ static void values(const char* from, uint32_t scale, u32x4_t (&x)[N / 4]) {
        const u32x4_t raw = *reinterpret_cast<const u32x4_t*>(from);
        if constexpr (E4M3) {
            x[0] = dequant8(u32x2_t{raw[0], raw[1]}, scale_of(scale));
            x[1] = dequant8(u32x2_t{raw[2], raw[3]}, scale_of(scale));
        } else {
            x[0] = raw;
        }
    }
    template <typename F>
    __device__ __forceinline__ static void each_token(const Kv& c, int32_t page, int32_t head, F use) {
        const int lane = threadIdx.x & 63, n = 1 << c.page_shift;
        const char* base = c.k + (E4M3 ? 1 : 2) * kv_off(c, page, head, 0) + 16 * (lane % LPT);
        const uint8_t* scales = c.k_scale + (E4M3 ? scale_off(c, page, head, 0) : 0);
        const int64_t step = (E4M3 ? 1 : 2) * c.token_stride;
        for (int t = lane / LPT; t < n; t += AHEAD * TOKENS) {
            u32x4_t x[AHEAD][N / 4];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int token = min(t + i * TOKENS, n - 1);  // the last one again changes nothing
                values(base + token * step, E4M3 ? scales[token] : 0, x[i]);
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) use(x[i]);
        }
    }
    __device__ __forceinline__ void find(const Kv& c, int32_t page, int32_t head) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            hi[j] = s16x2_t{-32768, -32768};
            lo[j] = s16x2_t{32767, 32767};
        }
        each_token(c, page, head, [&](const u32x4_t(&x)[N / 4]) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const s16x2_t y = ordered(__builtin_bit_cast(s16x2_t, (uint32_t)x[j / 4][j % 4]));
                hi[j] = __builtin_elementwise_max(hi[j], y);
                lo[j] = __builtin_elementwise_min(lo[j], y);
            }
        });
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int o = LPT; o < 64; o <<= 1) {
                hi[j] = __builtin_elementwise_max(
                    hi[j], __builtin_bit_cast(s16x2_t, __shfl_xor(__builtin_bit_cast(int, hi[j]), o)));
                lo[j] = __builtin_elementwise_min(
                    lo[j], __builtin_bit_cast(s16x2_t, __shfl_xor(__builtin_bit_cast(int, lo[j]), o)));
            }
    }
};

// Pages with infinities or NaN: the largest and smallest of what is not NaN, and
// the largest finite absolute value, element by element.
template <int D, bool E4M3, int E>
__device__ __forceinline__ uint32_t careful_bounds(const Kv& c, int32_t page, int32_t head, float (&hi)[E], float (&lo)[E]) {
    typedef PageBounds<D, E4M3> P;
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
        for (int o = P::LPT; o < 64; o <<= 1) {
            hi[j] = fmaxf(hi[j], __shfl_xor(hi[j], o));
            lo[j] = fminf(lo[j], __shfl_xor(lo[j], o));
        }
        if (hi[j] < lo[j]) hi[j] = lo[j] = 0.f;  // nothing but NaN
    }
    for (int o = 1; o < 64; o <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    return top;
}

template <int D, bool E4M3>
__global__ __launch_bounds__(256) void kv_bounds_kernel(BoundsArgs a) {
    typedef PageBounds<D, E4M3> P;
    constexpr int E = 2 * P::N;  // elements of a lane
    const int lane = threadIdx.x & 63;
    const int64_t units = (int64_t)a.n_pages * a.kv.n_kv_heads;
    for (int64_t u = (int64_t)blockIdx.x * 4 + wave_id(); u < units; u += (int64_t)gridDim.x * 4) {
        const int32_t page = clamp_page(a.kv, a.pages[u / a.kv.n_kv_heads]), head = (int32_t)(u % a.kv.n_kv_heads);
        P p;
        p.find(a.kv, page, head);
        float hi[E], lo[E];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < P::N; ++j) {
            const uint32_t h = __builtin_bit_cast(uint32_t, ordered(p.hi[j])), l = __builtin_bit_cast(uint32_t, ordered(p.lo[j]));
            hi[2 * j] = bf16_lo(h);
            hi[2 * j + 1] = bf16_hi(h);
            lo[2 * j] = bf16_lo(l);
            lo[2 * j + 1] = bf16_hi(l);
            top = max(max(top, max(h & 0x7FFFu, l & 0x7FFFu)), max(h >> 16 & 0x7FFFu, l >> 16 & 0x7FFFu));
        }
#pragma unroll
        for (int o = 1; o < P::LPT; o <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
        if (top >= 0x7F80u) top = careful_bounds<D, E4M3, E>(a.kv, page, head, hi, lo);
        const int e = code_exponent(top);
        const float unit = power(-e);
        const int64_t at = (int64_t)page * a.kv.n_kv_heads + head;
        if (lane < 2 * P::LPT) {  // the first token's lanes have the largest, the second's the smallest
            uint32_t w[E / 4];
#pragma unroll
            for (int j = 0; j < E; j += 4) {
                int x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = code(lane < P::LPT ? hi[j + i] : lo[j + i], unit);
                w[j / 4] = pack4(x[0], x[1], x[2], x[3]);
            }
            int8_t* to = a.codes + at * 2 * D + E * lane;
            if constexpr (E4M3) *reinterpret_cast<u32x4_t*>(to) = u32x4_t{w[0], w[1], w[2], w[3]};
            else *reinterpret_cast<u32x2_t*>(to) = u32x2_t{w[0], w[1]};
        }
        if (lane == 0) a.exps[at] = (uint8_t)(e + 127);
    }
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
    // tiles of 16 pages to score
    __device__ __forceinline__ int tiles(const SelectArgs& a) const {
        return a.select > a.first + a.last ? (scored(a, n - 1) + 15) >> 4 : 0;
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

// Scores are the products of a tile of 16 rows (query heads of one or more
// tokens) with 16 pages on the 8-bit matrix unit: sum max(r hi, r lo) =
// max(r, 0) . hi + min(r, 0) . lo.  As whole numbers they are exact; times their
// power of two they are below 2^121 and at least 2^-100, exact in fp32 as well.
template <int D>
struct Rows16 {
    static constexpr int S = D / 64;
    s32x4_t up[S], down[S];  // max(r, 0) and min(r, 0) of row lane % 16: elements 64 s + 16 (lane / 16) + 0..15

    __device__ __forceinline__ static int heads(const SelectArgs& a) { return (a.group + 15) >> 4; }  // tiles of a token
    __device__ __forceinline__ static const uint16_t* row(const SelectArgs& a, const SelectItem& it, int head, int tile,
                                                          int first) {
        const int r = threadIdx.x & 15, token = min(first + (r >> a.pad_shift), it.n - 1);
        const int h = min(16 * tile + (r & ((1 << a.pad_shift) - 1)), a.group - 1);  // the last head again changes no maximum
        return a.q + (it.row + token) * a.ldq + ((int64_t)head * a.group + h) * D + 16 * (threadIdx.x >> 4 & 3);
    }
    // tokens from `first` on of the item, heads of `tile`
    __device__ __forceinline__ void load(const SelectArgs& a, const SelectItem& it, int head, int tile, int first) {
        uint32_t top = 0;
        u32x4_t x[2 * S];
        const auto read = [&](int t) {
            const uint16_t* q = row(a, it, head, t, first);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                x[2 * s] = *reinterpret_cast<const u32x4_t*>(q + 64 * s);
                x[2 * s + 1] = *reinterpret_cast<const u32x4_t*>(q + 64 * s + 8);
            }
        };
        const int tiles = heads(a);
        for (int t = 1; t <= tiles; ++t) {  // the tile itself last
            read((tile + t) % tiles);
#pragma unroll
            for (int i = 0; i < 2 * S; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t lo = x[i][j] & 0x7FFFu, hi = x[i][j] >> 16 & 0x7FFFu;
                    top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
                }
        }
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        for (int o = 1; o < 1 << a.pad_shift; o <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
        const float unit = power(-code_exponent(top));
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w0 = x[2 * s + j / 2][2 * (j % 2)], w1 = x[2 * s + j / 2][2 * (j % 2) + 1];
                const int c0 = code(bf16_lo(w0), unit), c1 = code(bf16_hi(w0), unit);
                const int c2 = code(bf16_lo(w1), unit), c3 = code(bf16_hi(w1), unit);
                up[s][j] = (int)pack4(max(c0, 0), max(c1, 0), max(c2, 0), max(c3, 0));
                down[s][j] = (int)pack4(min(c0, 0), min(c1, 0), min(c2, 0), min(c3, 0));
            }
    }
};
template <int D>
struct Pages16 {
    static constexpr int S = D / 64;
    s32x4_t hi[S], lo[S];
    uint32_t exp;
    __device__ __forceinline__ void load(const SelectArgs& a, int32_t page, int head) {
        const int64_t at = (int64_t)min((uint32_t)page, (uint32_t)(a.n_pages - 1)) * a.n_kv_heads + head;
        const int8_t* p = a.codes + at * 2 * D + 16 * (threadIdx.x >> 4 & 3);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            hi[s] = *reinterpret_cast<const s32x4_t*>(p + 64 * s);
            lo[s] = *reinterpret_cast<const s32x4_t*>(p + D + 64 * s);
        }
        exp = a.exps[at];
    }
    __device__ __forceinline__ s32x4_t score(const Rows16<D>& r) const {
        s32x4_t x = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            x = __builtin_amdgcn_mfma_i32_16x16x64_i8(r.up[s], hi[s], x, 0, 0, 0);
            x = __builtin_amdgcn_mfma_i32_16x16x64_i8(r.down[s], lo[s], x, 0, 0, 0);
        }
        return x;
    }
};
// An unsigned number of the order of x.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}

// Keys of the item's scored pages, tiles of 16 pages from `tile` on in steps of
// `step`, for up to R tiles of rows at once; the bounds of AHEAD tiles are under
// way.  put(token, page, key, again) takes the keys, `again` where an earlier tile
// of heads has given one.  The same lane gives a page's key every time.
template <int D, int R, int AHEAD, typename Put>
__device__ __forceinline__ void score_pages(const SelectArgs& a, const SelectItem& it, int head, int tile, int step,
                                            int end, Put put) {
    const int col = threadIdx.x & 15, g = threadIdx.x >> 4 & 3, count = it.scored(a, it.n - 1), per = 16 >> a.pad_shift;
    const int32_t* table = it.table + a.first;
    for (int t = 0; t < Rows16<D>::heads(a); ++t) {
        if (tile >= end) return;
        Pages16<D> p[AHEAD];
        int32_t page[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) page[j] = table[min(16 * (tile + j * step) + col, count - 1)];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (tile + j * step < end) p[j].load(a, page[j], head);
            page[j] = table[min(16 * (tile + (j + AHEAD) * step) + col, count - 1)];
        }
        Rows16<D> r[R];
#pragma unroll
        for (int x = 0; x < R; ++x)
            if (x == 0 || x * per < it.n) r[x].load(a, it, head, t, x * per);
        for (int i = tile; i < end;) {
#pragma unroll
            for (int j = 0; j < AHEAD; ++j, i += step) {
                if (i >= end) break;
                s32x4_t score[R];
#pragma unroll
                for (int x = 0; x < R; ++x)
                    if (x == 0 || x * per < it.n) score[x] = p[j].score(r[x]);
                const float unit = scale_of(p[j].exp);
                if (i + AHEAD * step < end) p[j].load(a, page[j], head);
                page[j] = table[min(16 * (i + 2 * AHEAD * step) + col, count - 1)];
                const int at = 16 * i + col;
#pragma unroll
                for (int x = 0; x < R; ++x) {
                    if (x > 0 && x * per >= it.n) continue;
                    const auto give = [&](int token, int best) {
                        token += x * per;
                        if (token < it.n && at < count) put(token, at, key_of((float)best * unit), t > 0);
                    };
                    const s32x4_t y = score[x];
                    // rows 4 g + 0..3 of page `col` are here
                    if (a.pad_shift == 0) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) give(4 * g + k, y[k]);
                    } else if (a.pad_shift == 1) {
                        give(2 * g, max(y[0], y[1]));
                        give(2 * g + 1, max(y[2], y[3]));
                    } else {
                        int m = max(max(y[0], y[1]), max(y[2], y[3]));
                        if (a.pad_shift > 2) m = max(m, __shfl_xor(m, 16));
                        if (a.pad_shift > 3) m = max(m, __shfl_xor(m, 32));
                        if ((g & ((1 << (a.pad_shift - 2)) - 1)) == 0) give(g >> (a.pad_shift - 2), m);
                    }
                }
            }
        }
    }
}

// f(x, ...) over a wave's lanes by moves between them: the result of all lanes up
// to each (F, 0 or none as `none`), in lane 63 that of all.
template <typename F>
__device__ __forceinline__ int wave_scan(int x, int none, F f) {
#define SP_STEP(ctrl, rows) x = f(x, __builtin_amdgcn_update_dpp(none, x, ctrl, rows, 0xF, false))
    SP_STEP(0x111, 0xF);  // from 1, 2, 4 and 8 lanes before, within 16
    SP_STEP(0x112, 0xF);
    SP_STEP(0x114, 0xF);
    SP_STEP(0x118, 0xF);
    SP_STEP(0x142, 0xA);  // the last of 16 to the next 16, the last of 32 to the other 32
    SP_STEP(0x143, 0xC);
#undef SP_STEP
    return x;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    const int y = wave_scan((int)x, 0, [](int u, int v) { return (int)max((uint32_t)u, (uint32_t)v); });
    return (uint32_t)__builtin_amdgcn_readlane(y, 63);
}

template <int WAVES>
struct SelectScratch {
    uint32_t hist[256];
    uint32_t gt[WAVES], eq[WAVES];
};
template <int TEAM>
__device__ __forceinline__ void team_sync() {
    if constexpr (TEAM > 1) {
        __syncthreads();
    } else {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
}

// Writes the page ids of the k largest of n keys, the earlier among equals, in
// order.  A team of waves (all of a workgroup, or one) finds the k-th key digit by
// digit from the first bit in which the keys differ, by counting; then every wave
// goes through a part of them of its own.
template <int TEAM, typename Keys, typename Scratch>
__device__ __forceinline__ void take_largest(const Keys& key, int n, int k, const int32_t* pages, int32_t* out,
                                             Scratch& s) {
    const int lane = threadIdx.x & 63, wave = TEAM > 1 ? wave_id() : 0;
    const int self = 64 * wave + lane;
    uint32_t most = 0, least = 0xFFFFFFFFu;
    for (int i = self; i < n; i += 64 * TEAM) {
        const uint32_t x = key(i);
        most = max(most, x);
        least = min(least, x);
    }
    most = wave_max(most);
    least = ~wave_max(~least);
    if constexpr (TEAM > 1) {
        if (lane == 0) {
            s.gt[wave] = most;
            s.eq[wave] = least;
        }
        __syncthreads();
        for (int w = 0; w < TEAM; ++w) {
            most = max(most, s.gt[w]);
            least = min(least, s.eq[w]);
        }
    }
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
            for (int i = self; i < 256; i += 64 * TEAM) s.hist[i] = 0;
            team_sync<TEAM>();
            for (int i = self; i < n; i += 64 * TEAM) {
                const uint32_t x = key(i);
                if ((x & mask) == prefix) atomicAdd(&s.hist[x >> shift & 255u], 1u);
            }
            team_sync<TEAM>();
            // digits from the largest down, four to a lane
            int c[4], sum = 0;
            for (int j = 0; j < 4; ++j) sum += c[j] = (int)s.hist[255 - 4 * lane - j];
            const int upto = wave_scan(sum, 0, [](int u, int v) { return u + v; });
            const int at = __ffsll((unsigned long long)__ballot(upto >= want)) - 1;
            int above = upto - sum, digit = 255 - 4 * lane, count = c[0];
            for (int j = 1; j < 4; ++j)
                if (above + count < want) {
                    above += count;
                    count = c[j];
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
    const int part = TEAM > 1 ? (n + 64 * TEAM - 1) / (64 * TEAM) * 64 : n;
    const int begin = min(n, wave * part), end = min(n, begin + part);
    int taken = 0, equal = 0;
    if constexpr (TEAM > 1) {
        uint32_t gt = 0, eq = 0;
        for (int i = begin + lane; i < begin + (end - begin + 63) / 64 * 64; i += 64) {
            const uint32_t x = i < end ? key(i) & mask : 0;
            gt += __popcll(__ballot(i < end && x > prefix));
            eq += __popcll(__ballot(i < end && x == prefix));
        }
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
    for (int i = begin + lane; i < begin + (end - begin + 63) / 64 * 64; i += 64) {
        const uint32_t x = i < end ? key(i) & mask : 0;
        const bool same = i < end && x == prefix;
        const unsigned long long eq = __ballot(same);
        const bool take = (i < end && x > prefix) || (same && equal + __popcll(eq & before) < want);
        const unsigned long long all = __ballot(take);
        if (take) out[taken + __popcll(all & before)] = pages[i];
        taken += __popcll(all);
        equal += __popcll(eq);
    }
}

// Token i's row of the result.
template <int TEAM, typename Keys, typename Scratch>
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
    if (k > 0) take_largest<TEAM>(key, n, k, it.table + a.first, out + a.first, s);
}

// Scores in LDS, and the choice, in one: of a single token (ONE) by 16 waves, which
// have 190 KB of bounds under way between them, or of several by four, each of
// which chooses for tokens of its own.
template <int D, bool ONE>
__global__ __launch_bounds__(ONE ? 1024 : 256, ONE ? 4 : 2) void select_kernel(SelectArgs a) {
    constexpr int WAVES = ONE ? 16 : 4;
    extern __shared__ uint32_t keys[];
    __shared__ SelectScratch<WAVES> s[ONE ? 1 : WAVES];
    const int head = blockIdx.x % a.n_kv_heads, w = wave_id();
    SelectItem it;
    if (!load_select(a, blockIdx.x / a.n_kv_heads, it)) return;
    const int tiles = it.tiles(a);
    if (tiles > 0) {
        score_pages<D, ONE ? 1 : SP_ROW_TILES, ONE ? 2 : 1>(a, it, head, w, WAVES, tiles,
                                                            [&](int token, int page, uint32_t x, bool again) {
                                                                uint32_t& to = keys[token * a.max_scored + page];
                                                                to = again ? max(to, x) : x;
                                                            });
        __syncthreads();
    }
    if constexpr (ONE) {
        select_token<WAVES>(a, it, head, 0, [&](int page) { return keys[page]; }, s[0]);
    } else {
        for (int i = w; i < it.n; i += WAVES)
            select_token<1>(a, it, head, i, [&](int page) { return keys[i * a.max_scored + page]; }, s[w]);
    }
}

// The same for single tokens in two launches, by way of memory.
constexpr int kScoreTiles = 32;  // tiles of 16 pages of a workgroup, about
template <int D>
__global__ __launch_bounds__(256) void score_kernel(SelectArgs a) {
    const int head = blockIdx.x % a.n_kv_heads;
    SelectItem it;
    if (!load_select(a, blockIdx.x / a.n_kv_heads, it)) return;
    uint32_t* keys = a.keys + (int64_t)blockIdx.x * a.max_scored;
    score_pages<D, 1, 2>(a, it, head, blockIdx.y * 4 + wave_id(), gridDim.y * 4, it.tiles(a),
                         [&](int, int page, uint32_t x, bool again) { keys[page] = again ? max(keys[page], x) : x; });
}
__global__ __launch_bounds__(1024) void choose_kernel(SelectArgs a) {
    __shared__ SelectScratch<16> s;
    const int head = blockIdx.x % a.n_kv_heads;
    SelectItem it;
    if (!load_select(a, blockIdx.x / a.n_kv_heads, it)) return;
    const uint32_t* keys = a.keys + (int64_t)blockIdx.x * a.max_scored;
    select_token<16>(a, it, head, 0, [&](int page) { return keys[page]; }, s);
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
    BoundsArgs a{to_kv(*kv), bounds->codes, bounds->exps, L->attn.meta + L->info.off_fresh, L->info.n_fresh};
    typedef void (*fn_t)(BoundsArgs);
    static const fn_t fn[2][2] = {{kv_bounds_kernel<64, false>, kv_bounds_kernel<64, true>},
                                  {kv_bounds_kernel<128, false>, kv_bounds_kernel<128, true>}};
    const int64_t blocks = ((int64_t)a.n_pages * a.kv.n_kv_heads + 3) / 4;
    const hipError_t e = launch(fn[kv->head_dim == 128][kv->dtype == LORA_KV_E4M3],
                                dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), dim3(256),
                                reinterpret_cast<hipStream_t>(hip_stream), a);
    return e == hipSuccess ? LORA_OK : LORA_EHIP;
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
        if ((int64_t)S.n_items * hk > kMaxBlocks) return LORA_EINVAL;
        a.items = items;
        void* p[] = {&a};
        const bool one = S.item_tokens == 1;
        typedef void (*fn_t)(SelectArgs);
        static const fn_t fn[2][2] = {{select_kernel<64, false>, select_kernel<64, true>},
                                      {select_kernel<128, false>, select_kernel<128, true>}};
        const size_t lds = sizeof(uint32_t) * (size_t)S.max_scored * (size_t)S.item_tokens;
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(fn[d == 128][one]),
                                             dim3((unsigned)(S.n_items * hk)), dim3(one ? 1024 : 256), p, lds, stream);
        return e == hipSuccess ? LORA_OK : LORA_EHIP;
    }
    if (workspace_floats < I.workspace_floats) return LORA_ECAPACITY;
    if (!workspace || !aligned16(workspace)) return LORA_EINVAL;
    if (S.item_tokens != 1) return LORA_EINVAL;
    const int64_t per = (int64_t)S.max_scored * hk, slab = sp_slab(per, S.n_items);
    if (slab * per > I.workspace_floats || slab * hk > kMaxBlocks) return LORA_EINVAL;
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
