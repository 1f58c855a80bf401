// gfx950 kernels of the paged cache and the attention over it, and their C-ABI
// launchers.
//
//   write  k, v of the batch's new tokens into the cache's pages, q and k turned
//          by their positions' angles first
//   read   a batch's cached tokens back as bf16
//   attn   out_i = sum_j w_ij v_j, w_ij = exp(scale q_i . k_j) / sum, over the
//          tokens that row i sees
//
// Attention works on the transposed products S^T = K Q^T and O^T = V^T P^T, so
// that a query is a column of every MFMA: its running maximum and sum live in
// the lanes of that column, and S^T leaves the first product in the registers
// in which the second one takes P^T.  In the 32x32 result a lane of half h =
// lane / 32 holds rows 8b + 4h + 0..3 (b = 0..3) of its column; the second
// product's operand wants 8 reduction elements per lane, any 8 as long as V^T
// brings the same ones.  So slots 0..3 stand for tokens 8b + 4h + 0..3 and
// slots 4..7 for 8(b+1) + 4h + 0..3: the registers as they are.  The 16x16
// form works alike with tokens 4g + 0..3 and 16 + 4g + 0..3 of lane group g.
// V^T's fragments come out of row-major V tiles by transposing LDS reads
// (16 lanes read 4 rows x 16 columns, 8 bytes each, and get a column of 4).
//
// The scores are kept in base 2 (scale * log2 e is folded into one multiply-add)
// and the accumulator is rescaled only when a row's maximum grows by more than
// 2^8 over the one in use: weights then stay below 2^8, far inside fp32 and
// bf16, and the common tile pays neither the rescale nor a reduction over
// lanes (16 prompts of up to 2048 tokens take 113 us with a rescale at any
// growth where they take 108 so; 2 x 1024 tokens over 33k 1972 and 1904).
//
// Weights are rounded to bf16 for the second product, and the rounded weights are
// what the row's sum adds up, so the rounding cancels where few tokens dominate:
// the 4x4x4 MFMA with a first operand of ones gives each lane the sum of the four
// weights that it holds itself.  In the narrow kernel, which waits for memory, a
// second product adds what the rounding left (16 bits of a weight in all): outputs
// are then as exact as their own type, off by 1.7e-3 of their norm where one part
// gives 2.2e-3, for 0.2 us of a call.  In the wide one that takes 141 us where one
// part takes 104 (prompts) and 3342 for 1903 (long chunks): its outputs are off by
// 2.0e-3 to 2.4e-3.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "../../include/hetlora.h"
#define AT_FN static __host__ __device__ inline
#include "attn_rules.h"

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.0f;  // growth of a maximum (in powers of two) that is let pass
// A maximum m that is kept in base 2 is off by up to half a step from the score
// that it stands for, and all the row's weights by that power of two: 2^32 at
// most up to here.  Beyond, items are computed again from the scores' own
// differences (where a step of the scores is more than the weights can tell).
constexpr float kFar = 1073741824.0f;  // 2^30
// Weights of an item that is computed again are this much smaller, so that not
// even 2^30 of the largest values add up to infinity.  (Weights under 2^-90 of
// the row's largest are lost by it.)
constexpr float kCare = 2.3283064365386963e-10f;  // 2^-32

__device__ __forceinline__ f32x16_t mfma32(u32x4_t a, u32x4_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   c, 0, 0, 0);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// Two fp32 -> packed bf16, round to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const bf16x2_t p = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, p);
}
// l[0] += the four weights in w
__device__ __forceinline__ f32x4_t add_weights(uint32_t w0, uint32_t w1, f32x4_t l) {
    const u32x2_t ones = {0x3F803F80u, 0x3F803F80u}, w = {w0, w1};
    return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4_t, ones), __builtin_bit_cast(s16x4_t, w), l, 0,
                                                  0, 0);
}
// What a part of a row (a wave's or a split's: its output, maximum m and sum l)
// weighs where the row's maximum is top.  Outputs are joined as a weighted mean,
// which is no larger than they are.  A part with no maximum adds what it has:
// zeros where it saw nothing, NaN where every score that it saw was NaN.
__device__ __forceinline__ float part_weight(float m, float l, float top) {
    return m == -INFINITY ? l : l * __builtin_amdgcn_exp2f(m - top);
}
__device__ __forceinline__ float reciprocal(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Transposing LDS read: within each 16 lanes, lane i reads 8 bytes (4 bf16) and
// gets element i of the four 16-element rows that 4 lanes each supply.
__device__ __forceinline__ u32x2_t ds_tr16(const char* p) {
    typedef __attribute__((address_space(3))) s16x4_t lds_t;
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)p));
}

// ------------------------------------------------------------------ the cache
struct Kv {
    const char* k;
    const char* v;
    const uint8_t* k_scale;
    const uint8_t* v_scale;
    int64_t page_stride, head_stride, token_stride;
    int32_t n_pages, page_shift, n_kv_heads;
};
// A page id that is not one of the cache's (the host checks the table it
// stages) is read as the last page instead of outside the cache.
__device__ __forceinline__ int32_t clamp_page(const Kv& c, int32_t page) {
    return (int32_t)min((uint32_t)page, (uint32_t)(c.n_pages - 1));
}
__device__ __forceinline__ int64_t kv_off(const Kv& c, int32_t page, int32_t head, int32_t slot) {
    return page * c.page_stride + head * c.head_stride + slot * c.token_stride;
}
__device__ __forceinline__ int64_t scale_off(const Kv& c, int32_t page, int32_t head, int32_t slot) {
    return (((int64_t)page * c.n_kv_heads + head) << c.page_shift) + slot;
}
__device__ __forceinline__ float scale_of(uint32_t e) { return __uint_as_float(e << 23); }
// 8 e4m3 codes times a power of two -> 8 bf16 (exact)
__device__ __forceinline__ u32x4_t dequant8(u32x2_t c, float scale) {
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], scale, false));
        r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], scale, true));
    }
    return r;
}

// ------------------------------------------------------------------ write
struct WriteArgs {
    Kv kv;
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;
    const float* rope;
    uint16_t* q_out;
    int64_t ld_out;
    const int32_t* row_pos;
    const int32_t* row_slot;
    int32_t n_heads, n_vec, n_rows, rope_dim, rope_len;
};

template <bool F32>
__device__ __forceinline__ f32x4_t load4(const void* p, int64_t i) {
    if constexpr (F32) {
        return *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i);
    } else {
        const u32x2_t w = *reinterpret_cast<const u32x2_t*>(static_cast<const uint16_t*>(p) + i);
        return f32x4_t{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
    }
}
__device__ __forceinline__ float finite_abs(float x) {
    x = fabsf(x);
    return x < INFINITY ? x : 0.f;
}
// The e4m3 code of x * inv (inv a power of two), as lora_kv_t describes it.
__device__ __forceinline__ float e4m3_input(float x, float inv) {
    const float y = fminf(fmaxf(x * inv, -448.f), 448.f);
    return fabsf(x) < INFINITY ? y : __builtin_nanf("");
}

// D/8 lanes take one head's vector, 8 elements each: the pair elements c and c +
// rope_dim/2 of a turn lie in the same lane (4 and 4 of them), so nothing
// crosses lanes but the maximum.  The turn is written without multiply-adds:
// every product is rounded, as in the formula's plain evaluation in fp32, so
// that codes next to a rounding border do not depend on how it is evaluated.
// Bound by memory: 16 prompts of 128 to 2048 tokens (32 heads, fp32 in, e4m3
// cache) take 96 us, 5.8 TB/s; 64 single tokens 4 us, a launch.
template <int D, bool F32, bool E4M3>
__global__ __launch_bounds__(256) void kv_write_kernel(WriteArgs a) {
    constexpr int LPV = D / 8, VPB = 256 / LPV;
    const int row = blockIdx.y + gridDim.y * blockIdx.z;
    const int vec = blockIdx.x * VPB + threadIdx.x / LPV, i = threadIdx.x % LPV;
    if (row >= a.n_rows || vec >= a.n_vec) return;
    const int pos = a.row_pos[row], slot = a.row_slot[row];
    const int hk = a.kv.n_kv_heads;
    const bool is_q = vec < a.n_heads, is_k = !is_q && vec < a.n_heads + hk;
    const int head = is_q ? vec : is_k ? vec - a.n_heads : vec - a.n_heads - hk;
    const int half = a.rope_dim >> 1;
    const bool in_turn = 8 * i < a.rope_dim;
    const int c0 = in_turn ? 4 * i : 8 * i, c1 = in_turn ? half + 4 * i : 8 * i + 4;
    const void* src = is_q ? a.q : is_k ? a.k : a.v;
    const int64_t at = row * (is_q ? a.ldq : is_k ? a.ldk : a.ldv) + (int64_t)head * D;
    f32x4_t x = load4<F32>(src, at + c0), y = load4<F32>(src, at + c1);
    if (in_turn && (is_q || is_k) && pos >= 0 && pos < a.rope_len) {
#pragma clang fp contract(off)
        const f32x4_t c = *reinterpret_cast<const f32x4_t*>(a.rope + (int64_t)pos * a.rope_dim + c0);
        const f32x4_t s = *reinterpret_cast<const f32x4_t*>(a.rope + (int64_t)pos * a.rope_dim + c1);
        const f32x4_t u = x * c - y * s, w = x * s + y * c;
        x = u;
        y = w;
    }
    if (is_q) {
        uint16_t* o = a.q_out + row * a.ld_out + (int64_t)head * D;
        if (pos < 0) x = y = f32x4_t{0.f, 0.f, 0.f, 0.f};
        *reinterpret_cast<u32x2_t*>(o + c0) = u32x2_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
        *reinterpret_cast<u32x2_t*>(o + c1) = u32x2_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
        return;
    }
    const int32_t page = slot >> a.kv.page_shift;
    const bool held = slot >= 0 && page < a.kv.n_pages;
    const int32_t place = slot & ((1 << a.kv.page_shift) - 1);
    char* cache = const_cast<char*>(is_k ? a.kv.k : a.kv.v);
    if constexpr (!E4M3) {
        if (!held) return;
        uint16_t* o = reinterpret_cast<uint16_t*>(cache) + kv_off(a.kv, page, head, place);
        *reinterpret_cast<u32x2_t*>(o + c0) = u32x2_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
        *reinterpret_cast<u32x2_t*>(o + c1) = u32x2_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
    } else {
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, fmaxf(finite_abs(x[j]), finite_abs(y[j])));
#pragma unroll
        for (int o = 1; o < LPV; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
        // least e with top <= 1.75 * 2^8 * 2^e, from the bits of top = m * 2^t
        // (a subnormal top reads as t = -127, which the clamp covers)
        const uint32_t bits = __float_as_uint(top);
        int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        e = min(max(e, -100), 119);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t lo = 0, hi = 0;
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_input(x[0], inv), e4m3_input(x[1], inv), lo, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_input(x[2], inv), e4m3_input(x[3], inv), lo, true);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_input(y[0], inv), e4m3_input(y[1], inv), hi, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_input(y[2], inv), e4m3_input(y[3], inv), hi, true);
        if (!held) return;
        char* o = cache + kv_off(a.kv, page, head, place);
        *reinterpret_cast<uint32_t*>(o + c0) = lo;
        *reinterpret_cast<uint32_t*>(o + c1) = hi;
        uint8_t* sc = const_cast<uint8_t*>(is_k ? a.kv.k_scale : a.kv.v_scale);
        if (i == 0) sc[scale_off(a.kv, page, head, place)] = (uint8_t)(e + 127);
    }
}

// ------------------------------------------------------------------ read
struct ReadArgs {
    Kv kv;
    uint16_t *k_out, *v_out;
    int64_t ld;
    const int32_t* kv_start;
    const int32_t* table;
    int32_t n_seq, n_tokens, ld_table;
};

// D/8 lanes take one token and several heads: 8 elements of k and 8 of v of each.
// A workgroup finds the sequence of its first token by bisection, a lane goes on
// from there, and every head's loads are under way before the first is stored.
// Bound by memory: 48 sequences of up to 16384 tokens (8 kv heads, e4m3) take
// 171 us, 5.7 TB/s; eight heads a lane 174, stores that stay in the caches 186.
// (The first form, one head a lane with a bisection each, took 284.)
constexpr int kReadHeads = 4;
template <int D, bool E4M3>
__global__ __launch_bounds__(256) void kv_read_kernel(ReadArgs a) {
    constexpr int LPV = D / 8, VPB = 256 / LPV, HEADS = kReadHeads;
    typedef typename std::conditional<E4M3, u32x2_t, u32x4_t>::type raw_t;
    const int hk = a.kv.n_kv_heads, groups = (hk + HEADS - 1) / HEADS, c = 8 * (threadIdx.x % LPV);
    const int64_t n_blocks = ((int64_t)a.n_tokens + VPB - 1) / VPB * groups;
    for (int64_t block = blockIdx.x; block < n_blocks; block += gridDim.x) {
        const int first = (int)(block / groups) * VPB, head0 = (int)(block % groups) * HEADS;
        const int token = first + (int)threadIdx.x / LPV;
        if (token >= a.n_tokens) continue;
        int seq = 0, hi = a.n_seq;  // kv_start[seq] <= first < kv_start[seq + 1]
        while (hi - seq > 1) {
            const int mid = (seq + hi) >> 1;
            if (a.kv_start[mid] <= first) seq = mid;
            else hi = mid;
        }
        while (seq + 1 < a.n_seq && a.kv_start[seq + 1] <= token) ++seq;
        const int t = token - a.kv_start[seq];
        const int32_t page = clamp_page(a.kv, a.table[(int64_t)seq * a.ld_table + (t >> a.kv.page_shift)]);
        const int32_t place = t & ((1 << a.kv.page_shift) - 1);
        raw_t k[HEADS], v[HEADS];
        uint32_t ks[HEADS], vs[HEADS];
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            const int head = min(head0 + h, hk - 1);
            const int64_t off = (kv_off(a.kv, page, head, place) + c) * (E4M3 ? 1 : 2);
            if constexpr (E4M3) {
                const int64_t so = scale_off(a.kv, page, head, place);
                ks[h] = a.kv.k_scale[so];
                vs[h] = a.kv.v_scale[so];
            }
            k[h] = *reinterpret_cast<const raw_t*>(a.kv.k + off);
            v[h] = *reinterpret_cast<const raw_t*>(a.kv.v + off);
        }
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            if (head0 + h >= hk) break;
            const int64_t out = (int64_t)token * a.ld + (int64_t)(head0 + h) * D + c;
            u32x4_t x, y;
            if constexpr (E4M3) {
                x = dequant8(k[h], scale_of(ks[h]));
                y = dequant8(v[h], scale_of(vs[h]));
            } else {
                x = k[h];
                y = v[h];
            }
            __builtin_nontemporal_store(x, reinterpret_cast<u32x4_t*>(a.k_out + out));
            __builtin_nontemporal_store(y, reinterpret_cast<u32x4_t*>(a.v_out + out));
        }
    }
}

// ------------------------------------------------------------------ attention
struct AttnArgs {
    Kv kv;
    const lora_attn_work_t* work;
    const int32_t* table;
    const uint16_t* q;
    uint16_t* out;
    float* part;  // [n_kv_heads][part_rows][D] splits' outputs, then [n_kv_heads][part_rows][2] of (maximum, sum)
    int64_t ldq, ldo, part_rows;
    int32_t n_seq, n_rows, max_kv, ld_table, group, window, sinks;
    uint32_t inv_group;  // 2^31 / group, rounded up
    float sl2;  // scale * log2 e
};

// i / group for i < group + 256 (group up to AT_MAX_GROUP): the rounded-up
// reciprocal is less than 2^-31 too large, and i * group stays below 2^31.
__device__ __forceinline__ int token_of(const AttnArgs& a, int i) { return (int)__umulhi(2 * (uint32_t)i, a.inv_group); }
// What every lane of an item needs to know.
struct Item : lora_attn_work_t {
    int32_t p0;  // position of the first row's token
    const int32_t* table;
    AtSpan span;
};
// Items that do not lie inside the batch are skipped, so a corrupted work list
// cannot index outside the buffers.
__device__ __forceinline__ bool load_item(const AttnArgs& a, int i, int max_rows, bool merge, Item& it) {
    static_cast<lora_attn_work_t&>(it) = a.work[i];
    const int last_tok = token_of(a, it.lead + it.nrows - 1);
    if (!at_inside(&it, a.n_seq, a.n_rows, a.max_kv, a.group, max_rows, a.part_rows, last_tok, merge)) return false;
    it.p0 = it.kv - it.n_new + it.tok0;
    it.table = a.table + (int64_t)it.seq * a.ld_table;
    it.span = at_span(it.p0, it.p0 + last_tok, a.window, a.sinks);
    it.it0 = max(it.it0, 0);
    it.it1 = min(it.it1, merge ? it.nrows : at_span_tiles(it.span));
    return true;
}
// Position of the item's row r, and the element offset of its query or result
// (query head lead + r of the group, tokens on end, of kv head h).
__device__ __forceinline__ int row_pos(const AttnArgs& a, const Item& it, int r) { return it.p0 + token_of(a, it.lead + r); }
__device__ __forceinline__ int64_t row_off(const AttnArgs& a, const Item& it, int r, int h, int64_t ld, int D) {
    const int t = token_of(a, it.lead + r);
    return (int64_t)(it.q0 + it.tok0 + t) * ld + (int64_t)(h * a.group + it.lead + r - t * a.group) * D;
}
__device__ __forceinline__ bool sees(const AttnArgs& a, int pos, int token) {
    return token <= pos && (a.window == 0 || token > pos - a.window || token < a.sinks);
}
// Calls `each` with a function of e that says whether token `first` + e is hidden
// from the row at `pos`: once for what comes after the row and, with a window,
// once for what lies between the sinks and the window.  One comparison each, and
// one after the other: scheduled together, the comparisons' results took the
// scalar registers of the whole loop.
template <typename F>
__device__ __forceinline__ void hide(const AttnArgs& a, int pos, int first, F each) {
    const int left = pos - first;
    each([&](int e) {
        __builtin_amdgcn_sched_barrier(0);
        return e > left;
    });
    if (a.window) {
        const uint32_t from = (uint32_t)first - (uint32_t)a.sinks, count = (uint32_t)max(0, max(0, pos - a.window + 1) - a.sinks);
        each([&](int e) {
            __builtin_amdgcn_sched_barrier(0);
            return from + (uint32_t)e < count;
        });
    }
}
// Every row of positions p_lo .. p_hi sees all of tokens t0 .. t1; and: none sees any.
__device__ __forceinline__ bool all_see(const AttnArgs& a, int p_lo, int p_hi, int t0, int t1) {
    return t1 <= p_lo && (a.window == 0 || t0 > p_hi - a.window || t1 < a.sinks);
}
__device__ __forceinline__ bool none_sees(const AttnArgs& a, int p_lo, int p_hi, int t0, int t1) {
    return t0 > p_hi || (a.window != 0 && t1 <= p_lo - a.window && t0 >= a.sinks);
}

// Tiles in LDS are row-major bf16, D * 2 bytes a row, with the 16-byte chunks of
// a row permuted so that the lanes an LDS cycle serves (256 bytes) hit all banks
// once.  K: 16 lanes read one chunk of 16 rows.  V: 32 lanes read 32 bytes of 4
// rows of two neighbouring column blocks (wide) or of 8 rows (narrow); the row's
// low bits move the pair of chunks, and leave the pair's last bit to bit 2.
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c) {
    return c ^ (D == 128 ? row & 15 : (row >> 1) & 7);
}
template <int D>
__device__ __forceinline__ int v_chunk(int row, int c) {
    return c ^ ((D == 128 ? (row & 3) << 2 : (row & 2) << 1) | ((row >> 1) & 2));
}

// 16 bytes per lane from memory to LDS, past the registers: lane i's go to lds +
// 16 i.  They have arrived after wait_loads().  Written in assembly because the
// compiler, which cannot tell one half of LDS from the other behind the
// transposing reads, would wait for the next tile's copies before reading this
// one's; there is no register result that it could misplace.
__device__ __forceinline__ void copy_to_lds(const char* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
                 : "memory", "m0");
}
__device__ __forceinline__ void copy_to_lds(const char* from, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(from) : "memory", "m0");
}
// Until at most N of the wave's loads, the last ones, are under way.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Barrier of the workgroup that waits for LDS writes, not for loads.
__device__ __forceinline__ void barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ uint32_t lds_addr(const char* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// How NW waves move a tile of ROWS tokens: a wave moves RPI rows at a time, 16
// bytes of bf16 (or 8 of codes) per lane, in STEPS steps.
template <int D, int NW, int ROWS>
struct Split {
    static constexpr int CPR = D / 8, RPI = 64 / CPR, STEPS = ROWS / (RPI * NW);
    // first row of step s of a wave
    static __device__ __forceinline__ int row(int s, int wave) { return (s * NW + wave) * RPI; }
};

// Where a wave's rows of the item's tiles lie in the cache: addresses of their
// keys.  `Tiles` maps a tile's number to its first token; numbers past the last
// tile stand for it.  Tokens past the end of the sequence take its last token's
// place: nothing sees them.
//
// UNI: a page holds RPI tokens at least, so a step's rows lie in one page, and the
// address is that of their first row.  Each lane works out the address of one
// step of one of the next 64 / STEPS tiles, from a page id fetched a window
// earlier; a tile then only reads lanes.  (Looked up tile by tile with scalar
// loads and multiplies, the same took longer than the tile's softmax: a scalar
// instruction that waits for another takes ten cycles.)  Otherwise every lane
// looks up the page of its own row, tile by tile: 113 us where this takes 108 (16
// prompts of up to 2048 tokens), 2007 for 1904 (2 x 1024 tokens over 33k).
template <int D, bool E4M3, bool UNI, int NW, int ROWS, typename Tiles>
struct Places {
    typedef Split<D, NW, ROWS> S;
    typedef typename std::conditional<UNI, uint32_t, int64_t>::type scale_t;
    static constexpr int STEPS = S::STEPS, WINDOW = 64 / STEPS, ES = E4M3 ? 1 : 2;
    const Kv& c;
    const Item& it;
    const Tiles& tiles;
    const uint64_t base;  // the head's first key
    const int wave, lane;
    int32_t ahead[UNI ? 1 : STEPS];  // page ids looked up
    uint32_t lo, hi, so, more;  // UNI, a step a lane: address, scale offset, rows after the first (at most RPI - 1)
    // of the tile last asked for: address and scale offset of the step's first row (UNI) or of the lane's row
    uint64_t at[STEPS];
    scale_t sc[STEPS];
    uint32_t rows[UNI ? STEPS : 1];

    __device__ __forceinline__ Places(const Kv& c_, const Item& it_, const Tiles& tiles_, int head, int wave_)
        : c(c_), it(it_), tiles(tiles_), base((uint64_t)(uintptr_t)c_.k + ES * head * c_.head_stride), wave(wave_),
          lane(threadIdx.x & 63) {}
    __device__ __forceinline__ int window_token(int i) const { return tiles(i + lane / STEPS) + S::row(lane % STEPS, wave); }
    __device__ __forceinline__ int token(int i, int s) const {
        return min(tiles(i) + S::row(s, wave) + lane / S::CPR, it.kv - 1);
    }
    // UNI: the pages of the window that starts at tile i; else of tile i
    __device__ __forceinline__ void look_up(int i) {
        if constexpr (UNI) {
            ahead[0] = it.table[min(window_token(i), it.kv - 1) >> c.page_shift];
        } else {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) ahead[s] = it.table[token(i, s) >> c.page_shift];
        }
    }
    // Tile i is the next to be asked for; tiles are asked for in order, from 0,
    // after look_up(0).
    __device__ __forceinline__ void open(int i) {
        if (!UNI || i % WINDOW != 0) return;
        const int first = window_token(i), tok = min(first, it.kv - 1);
        const int32_t pg = clamp_page(c, ahead[0]), slot = tok & ((1 << c.page_shift) - 1);
        const uint64_t x = base + ES * ((uint64_t)(uint32_t)pg * (uint32_t)c.page_stride +
                                        (uint64_t)(uint32_t)slot * (uint32_t)c.token_stride);
        lo = (uint32_t)x;
        hi = (uint32_t)(x >> 32);
        so = (uint32_t)(((uint32_t)pg * (uint32_t)c.n_kv_heads << c.page_shift) + slot);
        more = (uint32_t)min(max(it.kv - 1 - first, 0), S::RPI - 1);
        look_up(i + WINDOW);
    }
    __device__ __forceinline__ void read(int i) {
        if constexpr (UNI) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int l = (i % WINDOW) * STEPS + s;
                at[s] = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, l) << 32) |
                        (uint32_t)__builtin_amdgcn_readlane(lo, l);
                rows[s] = __builtin_amdgcn_readlane(more, l);
                if constexpr (E4M3) sc[s] = __builtin_amdgcn_readlane(so, l);
            }
        } else {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int32_t pg = clamp_page(c, ahead[s]), slot = token(i, s) & ((1 << c.page_shift) - 1);
                at[s] = base + ES * (pg * c.page_stride + slot * c.token_stride);
                if constexpr (E4M3) sc[s] = scale_off(c, pg, 0, slot);
            }
            look_up(i + 1);
        }
    }
};

// Keys (or VALUES) of a tile on their way from the cache to LDS.  DIRECT: bf16
// rows go straight to LDS, the permutation of a row's chunks made by the lanes'
// source addresses.  Otherwise they go through registers, and e4m3 codes become
// bf16 (exactly) on the way.
template <int D, bool E4M3, bool UNI, bool DIRECT, bool VALUES, int NW, int ROWS>
struct Stage {
    static_assert(!(E4M3 && DIRECT), "codes are converted on the way");
    typedef Split<D, NW, ROWS> S;
    static constexpr int STEPS = S::STEPS, ES = E4M3 ? 1 : 2, HELD = DIRECT ? 1 : STEPS;
    typedef typename std::conditional<E4M3, u32x2_t, u32x4_t>::type raw_t;
    typedef typename std::conditional<UNI, uint32_t, int64_t>::type scale_t;
    uint64_t at[STEPS];  // as in Places
    scale_t sc[STEPS];
    uint32_t rows[UNI ? STEPS : 1];
    const uint8_t* scales;  // the head's first scale
    uint64_t apart;         // values from keys
    int32_t wave;
    uint32_t row_bytes;
    raw_t held[HELD];
    uint32_t exps[E4M3 ? STEPS : 1];

    __device__ __forceinline__ void init(const Kv& c, int head, int wave_) {
        scales = (VALUES ? c.v_scale : c.k_scale) + ((int64_t)head << c.page_shift);
        apart = VALUES ? (uint64_t)(uintptr_t)c.v - (uint64_t)(uintptr_t)c.k : 0;
        wave = wave_;
        row_bytes = (uint32_t)c.token_stride * ES;
    }
    template <typename P>
    __device__ __forceinline__ void take(const P& p) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            at[s] = p.at[s] + apart;
            if constexpr (UNI) rows[s] = p.rows[s];
            if constexpr (E4M3) sc[s] = p.sc[s];
        }
    }
    __device__ __forceinline__ int chunk(int row) const {
        const int c = (threadIdx.x & 63) % S::CPR;
        return VALUES ? v_chunk<D>(row, c) : k_chunk<D>(row, c);
    }
    __device__ __forceinline__ void load(char* tile) {
        const int lane = threadIdx.x & 63, mine = lane / S::CPR;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const char* from = (const char*)(uintptr_t)at[s];
            uint32_t off = (DIRECT ? chunk(S::row(s, wave) + mine) : lane % S::CPR) * 8 * ES;
            if constexpr (UNI) off += min(mine * row_bytes, rows[s] * row_bytes);
            if constexpr (DIRECT) {
                const uint32_t to = lds_addr(tile) + S::row(s, wave) * (2 * D);
                if constexpr (UNI) copy_to_lds(from, off, to);
                else copy_to_lds(from + off, to);
            } else {
                held[s] = *reinterpret_cast<const raw_t*>(from + off);
            }
            if constexpr (E4M3) {
                if constexpr (UNI) exps[s] = scales[sc[s] + min((uint32_t)mine, rows[s])];
                else exps[s] = scales[sc[s]];
            }
        }
    }
    // what load() has left in registers
    __device__ __forceinline__ void store(char* tile) const {
        if constexpr (!DIRECT) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int row = S::row(s, wave) + (threadIdx.x & 63) / S::CPR;
                u32x4_t x;
                if constexpr (E4M3) x = dequant8(held[s], scale_of(exps[s]));
                else x = held[s];
                *reinterpret_cast<u32x4_t*>(tile + row * (2 * D) + 16 * chunk(row)) = x;
            }
        }
    }
};

__device__ __forceinline__ float v_elem(const char* vt, int row_bytes, int row, int chunk, int e) {
    return __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t*>(vt + row * row_bytes + 16 * chunk + 2 * e)
                           << 16);
}

// One wave's rows in the wide kernel, and what it has of them so far.
template <int D>
struct Wide {
    int row, pos, p_lo, p_hi;  // this lane's row and its position; the wave's first and last position
    bool active;
    int whole0, whole1, whole2;  // every row sees all of tiles i < whole0 and whole1 <= i < whole2
    u32x4_t qf[D / 16];
    f32x16_t s[2];       // scores of a tile: S^T, 64 tokens x 32 rows
    uint32_t pw[16];     // its weights, in pairs
    f32x16_t acc[D / 32];  // O^T
    float m;
    f32x4_t l;  // the sum of the lane's weights, four times

    __device__ __forceinline__ void find_whole(const AttnArgs& a, const Item& it) {
        const int behind = at_max(0, (p_lo + 1) >> 6);  // tiles that end before the first row's next token
        const int list = it.span.sinks - it.span.first - it.it0;  // tile -> number, past the sinks
        whole0 = a.window ? min(min(a.sinks >> 6, behind), it.span.sinks) - it.it0 : 0;
        whole1 = a.window ? (at_max(-64, p_hi - a.window) >> 6) + 1 + list : 0;
        whole1 = max(whole1, it.span.sinks - it.it0);
        whole2 = behind + list;
    }
    __device__ __forceinline__ bool masks(int i) const { return !(i < whole0 || (i >= whole1 && i < whole2)); }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int d = 0; d < D / 32; ++d) acc[d] = f32x16_t{};
        m = -INFINITY;
        l = f32x4_t{};
    }
    // Operands of the multiplications in their order: chunk f / 2 of the keys'
    // tokens 32 (f % 2) ..., and 32 columns f % (D/32) of 16 tokens of the values.
    __device__ __forceinline__ static u32x4_t k_part(const char* kt, int f) {
        const int col = threadIdx.x & 31, h = (threadIdx.x >> 5) & 1, r = 32 * (f & 1) + col;
        return *reinterpret_cast<const u32x4_t*>(kt + r * (2 * D) + 16 * k_chunk<D>(r, 2 * (f >> 1) + h));
    }
    __device__ __forceinline__ static u32x4_t v_part(const char* vt, int f) {
        const int lane = threadIdx.x & 63, h = lane >> 5, i16 = lane & 15, g = (lane >> 4) & 1;
        const int r = 16 * (f / (D / 32)) + 4 * h + (i16 >> 2);
        const int ch = 4 * (f % (D / 32)) + 2 * g + ((i16 & 3) >> 1), by = 8 * (i16 & 1);
        const u32x2_t lo = ds_tr16(vt + r * (2 * D) + 16 * v_chunk<D>(r, ch) + by);
        const u32x2_t hi = ds_tr16(vt + (r + 8) * (2 * D) + 16 * v_chunk<D>(r + 8, ch) + by);
        return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
    }
    // Scores of one tile (SCORES) and product of another (PRODUCT).  LDS answers
    // after four MFMAs' time, so the operands are read AHEAD of them.
    template <bool SCORES, bool PRODUCT>
    __device__ __forceinline__ void multiply(const char* kt, const char* vt) {
        constexpr int NS = SCORES ? D / 8 : 0, N = NS + (PRODUCT ? D / 8 : 0), AHEAD = 6;
        u32x4_t part[AHEAD];
        const auto read = [&](int f) { return f < NS ? k_part(kt, f) : v_part(vt, f - NS); };
        if (SCORES) s[0] = s[1] = f32x16_t{};
#pragma unroll
        for (int f = 0; f < AHEAD; ++f) part[f] = read(f);
#pragma unroll
        for (int f = 0; f < N; ++f) {
            if (f < NS) {
                s[f & 1] = mfma32(part[f % AHEAD], qf[f >> 1], s[f & 1]);
            } else {
                const int c = (f - NS) / (D / 32), d = (f - NS) % (D / 32);
                const u32x4_t pf = {pw[4 * c], pw[4 * c + 1], pw[4 * c + 2], pw[4 * c + 3]};
                acc[d] = mfma32(part[f % AHEAD], pf, acc[d]);
                if (d < 2) l = add_weights(pf[2 * d], pf[2 * d + 1], l);
            }
            if (f + AHEAD < N) part[f % AHEAD] = read(f + AHEAD);
            __builtin_amdgcn_sched_barrier(0x6);  // arithmetic may move
        }
    }
    // of tile i; CAREFUL: m is a score, not yet in base 2
    template <bool CAREFUL, typename Tiles>
    __device__ __forceinline__ void weights(const AttnArgs& a, const Tiles& tiles, int i) {
        const int h = (threadIdx.x >> 5) & 1;
        if (masks(i)) hide(a, pos, tiles(i) + 4 * h, [&](auto hidden) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (hidden(32 * b + 8 * (r >> 2) + (r & 3))) s[b][r] = -INFINITY;
        });
        float top = s[0][0];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
        const float unit = CAREFUL ? 1.f : a.sl2;  // of m
        if (__ballot(top * unit > m + (CAREFUL ? 0.f : kGrow))) {
            const float up = fmaxf(m, fmaxf(top, __shfl_xor(top, 32)) * unit);
            const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(CAREFUL ? (m - up) * a.sl2 : m - up);
            m = up;
            l *= f;
#pragma unroll
            for (int d = 0; d < D / 32; ++d) acc[d] *= f;
        }
        const float off = m == -INFINITY ? 0.f : -m;
        const auto weight = [&](float x) {
            if (CAREFUL) return kCare * __builtin_amdgcn_exp2f((x + off) * a.sl2);
            return __builtin_amdgcn_exp2f(fmaf(x, a.sl2, off));
        };
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; r += 2) pw[8 * b + r / 2] = pack_bf16(weight(s[b][r]), weight(s[b][r + 1]));
    }
    // the product of each row's visible tokens alone
    __device__ __forceinline__ void careful_product(const AttnArgs& a, const char* vt, int t0) {
        const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
        // one pair of rows' weights after the other, each register moved down
        // to the first: a rolled loop over registers
#pragma unroll 1
        for (int j = 0; j < 16; ++j) {
            const uint32_t cur = pw[0];
            l = add_weights(cur, 0, l);
#pragma unroll
            for (int k = 0; k < 15; ++k) pw[k] = pw[k + 1];
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
                const uint32_t both = __shfl(cur, col + 32 * (x >> 1));
                const float p = x & 1 ? bf16_hi(both) : bf16_lo(both);
                const int r = 2 * (j & 7) + (x & 1);
                const int tok = 32 * (j >> 3) + 8 * (r >> 2) + 4 * (x >> 1) + (r & 3);
                const bool vis = sees(a, pos, t0 + tok);
#pragma unroll
                for (int d = 0; d < D / 32; ++d)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int el = 32 * d + 8 * (e >> 2) + 4 * h + (e & 3);
                        const float v = v_elem(vt, 2 * D, tok, v_chunk<D>(tok, el >> 3), el & 7);
                        acc[d][e] = vis ? fmaf(p, v, acc[d][e]) : acc[d][e];
                    }
            }
        }
    }
    // the rows' output; of a split with its maximum and sum (l is `unit` of it)
    __device__ __forceinline__ void finish(const AttnArgs& a, const Item& it, int head, bool mine, float unit) const {
        const int h = (threadIdx.x >> 5) & 1;
        const float total = l[0] + __shfl_xor(l[0], 32);
        if (!mine) return;
        const float inv = reciprocal(total);
        if (it.nsplits == 1) {
            // a lane's 4 elements and those of the other half's lane make 16 bytes
            uint16_t* o = a.out + row_off(a, it, row, head, a.ldo, D) + 8 * h;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int b = 0; b < 4; b += 2) {
                    u32x4_t out;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const f32x16_t& x = acc[d];
                        const auto both = __builtin_amdgcn_permlane32_swap(
                            pack_bf16(x[4 * b + 2 * e] * inv, x[4 * b + 2 * e + 1] * inv),
                            pack_bf16(x[4 * b + 2 * e + 4] * inv, x[4 * b + 2 * e + 5] * inv), false, false);
                        out[e] = both[0];
                        out[2 + e] = both[1];
                    }
                    *reinterpret_cast<u32x4_t*>(o + 32 * d + 8 * b) = out;
                }
        } else {
            const int64_t pr = head * a.part_rows + it.part + row;
            float* o = a.part + pr * D + 4 * h;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    *reinterpret_cast<f32x4_t*>(o + 32 * d + 8 * b) =
                        f32x4_t{acc[d][4 * b] * inv, acc[d][4 * b + 1] * inv, acc[d][4 * b + 2] * inv, acc[d][4 * b + 3] * inv};
            if (h == 0) {
                float* ml = a.part + (int64_t)a.kv.n_kv_heads * a.part_rows * D + 2 * pr;
                ml[0] = m;
                ml[1] = total / unit;
            }
        }
    }
    // The compiler may not move the multiplications, or the weights, past here: a
    // barrier alone orders memory, not registers.
    __device__ __forceinline__ void multiplied() {
#pragma unroll
        for (int b = 0; b < 2; ++b) asm volatile("" : "+v"(s[b]));
#pragma unroll
        for (int d = 0; d < D / 32; ++d) asm volatile("" : "+v"(acc[d]));
    }
    __device__ __forceinline__ void weighed() {
#pragma unroll
        for (int i = 0; i < 16; ++i) asm volatile("" : "+v"(pw[i]));
    }
    // The result is not finite, or its maximum is too far from zero: compute it with care.
    __device__ __forceinline__ bool needs_care() const {
        float bad = fabsf(m) >= kFar && m != -INFINITY ? 1.f : 0.f;
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) bad = fmaf(acc[d][e], 0.f, bad);
        return active && bad != 0.f;
    }
};

// Tile number -> first token, for a workgroup that takes all of the item's tiles.
// Numbers past the last one stand for the last.
struct AllTiles {
    AtSpan span;
    int32_t it0, last;
    __device__ __forceinline__ int operator()(int i) const { return AT_TILE * at_span_tile(span, min(it0 + i, last)); }
};

// A wave has 32 rows.  A tile of 64 tokens of 128 elements is 32 MFMAs for it
// (1024 cycles of the matrix unit) and about as many cycles of vector
// instructions (64 elements: 512 and as many): bound by the matrix unit where
// the two overlap.  2 x 1024 tokens of 64 heads over 33k (pair) take 1803 to 1907
// us, by card: 1230 to 1165 TFLOP/s of the 1530 that a large library product
// reaches; 16 prompts of up to 2048 tokens of 32 heads (wide) 101 to 109 us, 560
// to 520 TFLOP/s of what rows see:
// there an item has 7 tiles on average, and its start and end (work item, page
// ids and queries one after the other, the waves' different last tiles, the
// result) take as long as three.
//
// PAIR: eight waves, 256 rows.  Each SIMD has one wave of either half, and they
// alternate: between two barriers one half multiplies (the scores of its tile i
// and the product of tile i - 1) while the other one is at its softmax.  Left to
// themselves the two waves of a SIMD fell into step and took turns at both units.
// Otherwise four waves, 128 rows, and two workgroups to a compute unit, whose
// waves find gaps of each other's (the plan has both sides' times).
//
// Keys and values have NB tiles each in LDS.  Keys i + LEAD and values i + LEAD - 1
// are sent for in the softmax of tile i, into the place of tiles that every wave
// is done with; a wave waits for its own share of keys i + 1 and values i at the
// barrier before the first half multiplies them.  Past the last tile it is sent
// for again, which no one reads: a wave's loads in flight are then always as many.
//
// A value that is infinite or NaN in a place that a row does not see would
// still reach it through the second product (0 * NaN).  Looking for such values
// in every masked tile costs more than it is worth, so the item looks at its
// result: when that is not finite, it is computed again, and the tiles in which
// some row is masked take each row's visible tokens alone.  So are items whose
// maximum is kFar or more from zero.
template <int D, bool E4M3, bool UNI, bool PAIR>
__global__ __launch_bounds__(PAIR ? 512 : 256, 2) void attn_wide_kernel(AttnArgs a) {
    constexpr int BYTES = AT_TILE * 2 * D, NW = PAIR ? 8 : 4, NB = PAIR ? 4 : 2, LEAD = 3;
    constexpr bool DIRECT = !E4M3;
    typedef Stage<D, E4M3, UNI, DIRECT, false, NW, AT_TILE> KStage;
    typedef Stage<D, E4M3, UNI, DIRECT, true, NW, AT_TILE> VStage;
    constexpr int BOTH = KStage::STEPS + VStage::STEPS;  // loads of a wave for a tile's keys and values
    __shared__ __align__(16) char lds[2][NB][BYTES];
    const int head = blockIdx.x % a.kv.n_kv_heads, lane = threadIdx.x & 63, w = wave_id();
    const int col = lane & 31, h = lane >> 5;
    [[maybe_unused]] const bool second = PAIR && w >= 4;
    Item it;
    if (!load_item(a, blockIdx.x / a.kv.n_kv_heads, 32 * NW, false, it)) return;

    Wide<D> x;
    x.row = min(32 * w + col, it.nrows - 1);  // lanes past the item's rows repeat its last one
    x.active = 32 * w < it.nrows;
    x.pos = row_pos(a, it, x.row);
    x.p_lo = row_pos(a, it, min(32 * w, it.nrows - 1));
    x.p_hi = row_pos(a, it, min(32 * w + 31, it.nrows - 1));
    {
        const uint16_t* q = a.q + row_off(a, it, x.row, head, a.ldq, D) + 8 * h;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) x.qf[s] = *reinterpret_cast<const u32x4_t*>(q + 16 * s);
    }
    const int n = it.it1 - it.it0;
    if (n <= 0) {  // the rows see nothing
        x.clear();
        x.finish(a, it, head, 32 * w + col < it.nrows, 1.f);
        return;
    }
    const AllTiles tile{it.span, it.it0, it.it1 - 1};
    const auto keys = [&](int i) { return lds[0][i % NB]; };
    const auto values = [&](int i) { return lds[1][i % NB]; };
    KStage ks;
    VStage vs;
    ks.init(a.kv, head, w);
    vs.init(a.kv, head, w);
    Places<D, E4M3, UNI, NW, AT_TILE, AllTiles> places(a.kv, it, tile, head, w);
    x.find_whole(a, it);
    x.clear();
    places.look_up(0);
    // the queries arrive here: a wait for them inside the loop over tiles would
    // be one for the copies that are under way there
#pragma unroll
    for (int s = 0; s < D / 16; ++s) asm volatile("" : "+v"(x.qf[s]));
    if constexpr (!PAIR) {
        // Tile i's keys and values arrive together, behind the work on tile i - 1.
        const auto send = [&](int i) {
            places.open(i);
            places.read(i);
            ks.take(places);
            vs.take(places);
            ks.load(keys(i));
            vs.load(values(i));
        };
        send(0);
        for (int i = 0; i < n; ++i) {
            ks.store(keys(i));
            vs.store(values(i));
            if (DIRECT) wait_loads<0>();
            barrier();
            if (i + 1 < n) send(i + 1);
            const int t0 = tile(i);
            if (!x.active || none_sees(a, x.p_lo, x.p_hi, t0, t0 + AT_TILE - 1)) continue;
            x.template multiply<true, false>(keys(i), nullptr);
            x.template weights<false>(a, tile, i);
            x.template multiply<false, true>(nullptr, values(i));
        }
    } else {
        // values i + LEAD - 1 lie where keys i + LEAD - 1 did
        const auto plan = [&](int i) {
            if (i + LEAD > 0) vs.take(places);
            places.read(i + LEAD);
            ks.take(places);
        };
        const auto send_values = [&](int i) {
            if (i + LEAD > 0) vs.load(values(i + LEAD - 1));
        };
        const auto send_keys = [&](int i) { ks.load(keys(i + LEAD)); };
        // codes sent for the last time, into LDS
        const auto unpack = [&](int i) {
            if (DIRECT || i == -LEAD) return;
            if (i + LEAD > 1) vs.store(values(i + LEAD - 2));
            ks.store(keys(i + LEAD - 1));
        };
#pragma unroll
        for (int i = -LEAD; i < 0; ++i) {
            places.open(i + LEAD);
            plan(i);
            unpack(i);
            send_values(i);
            send_keys(i);
        }
        places.open(LEAD);
        wait_loads<DIRECT ? (LEAD - 1) * BOTH : 0>();
        barrier();
        if (second) barrier();
        const auto phase = [&](int i) {
            x.multiplied();
            __builtin_amdgcn_s_setprio(0);
            barrier();
            unpack(i);
            plan(i);
            send_values(i);
            send_keys(i);
            places.open(i + 1 + LEAD);
            x.template weights<false>(a, tile, i);
            x.weighed();
            if (DIRECT && !second) wait_loads<(LEAD - 1) * BOTH>();
            barrier();
            __builtin_amdgcn_s_setprio(1);  // the matrix unit goes first
        };
        const auto arrive = [&] {  // this half has not sent for the next tile's yet
            if (DIRECT && second) wait_loads<(LEAD - 2) * BOTH>();
        };
        x.template multiply<true, false>(keys(0), nullptr);
        arrive();
        int i = 0;
        for (; i < n - 1; ++i) {
            phase(i);
            x.template multiply<true, true>(keys(i + 1), values(i));
            arrive();
        }
        phase(i);
        x.template multiply<false, true>(nullptr, values(i));
        wait_loads<0>();
        if (!second) barrier();
    }

    float unit = 1.f;
    if (__syncthreads_or(x.needs_care())) {
        unit = kCare;
        x.clear();
        places.look_up(0);
        int i = 0;
        do {
            places.open(i);
            places.read(i);
            ks.take(places);
            vs.take(places);
            ks.load(keys(0));
            vs.load(values(0));
            ks.store(keys(0));
            vs.store(values(0));
            wait_loads<0>();
            barrier();
            x.template multiply<true, false>(keys(0), nullptr);
            x.template weights<true>(a, tile, i);
            if (x.masks(i)) x.careful_product(a, values(0), tile(i));
            else x.template multiply<false, true>(nullptr, values(0));
            barrier();
        } while (++i < n);
        x.m *= a.sl2;
    }

    x.finish(a, it, head, 32 * w + col < it.nrows, unit);
}

// Tile number -> first token of the tiles of 32 that one of the narrow kernel's
// four waves takes.
struct EveryFourth {
    AtSpan span;
    int32_t first, last;
    __device__ __forceinline__ int operator()(int i) const {
        const int x = min(first + 4 * i, last);
        return AT_TILE * at_span_tile(span, x >> 1) + 32 * (x & 1);
    }
};

// The narrow kernel's V tiles: v_chunk's order, and bit 3 of the row turns a
// pair's chunks, so that 16 lanes that write one chunk of 16 rows hit all banks.
template <int D>
__device__ __forceinline__ int n_chunk(int row, int c) {
    return v_chunk<D>(row, c) ^ ((row >> 3) & 1);
}

// One wave's tiles in the narrow kernel; true where the result needs care, as in Wide.
//
// Lane (col, g) = (lane % 16, lane / 16) loads parts of tokens col and 16 + col,
// of keys and values alike, at the addresses that it works out itself: 64 bytes
// of a token go to the 4 lanes of one load.  The keys are the first product's
// operand as they are loaded, with EPL elements in a row for each lane; q is
// loaded in the same order (q_part).  Only the values pass through LDS, which
// transposes them.
template <int D, bool E4M3>
struct NarrowTile {
    static constexpr int ES = E4M3 ? 1 : 2, EPL = 16 / ES, J = D / (4 * EPL), H = EPL / 8;
    // first element of operand k of lanes g
    static __device__ __forceinline__ int q_part(int k, int g) { return 4 * EPL * (k / H) + EPL * g + 8 * (k % H); }
    // operand k from a token's loads
    static __device__ __forceinline__ u32x4_t part(const u32x4_t (&raw)[J], uint32_t exp, int k) {
        const u32x4_t x = raw[k / H];
        if constexpr (E4M3) return dequant8(u32x2_t{x[2 * (k % H)], x[2 * (k % H) + 1]}, scale_of(exp));
        else return x;
    }
    u32x4_t k[2][J], v[2][J];
    uint32_t k_exp[2], v_exp[2];
    int32_t page[2];
    int64_t at[2], sc[2];  // bytes from the head's first token; scale

    __device__ __forceinline__ static int token(const Item& it, int t0, int b) {
        return min(t0 + 16 * b + (int)(threadIdx.x & 15), it.kv - 1);
    }
    __device__ __forceinline__ void look_up(const Kv& c, const Item& it, int t0) {
#pragma unroll
        for (int b = 0; b < 2; ++b) page[b] = it.table[token(it, t0, b) >> c.page_shift];
    }
    // of the tile that look_up() was last called for
    __device__ __forceinline__ void place(const Kv& c, const Item& it, int t0, int head) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int32_t pg = clamp_page(c, page[b]), slot = token(it, t0, b) & ((1 << c.page_shift) - 1);
            at[b] = ES * (pg * c.page_stride + slot * c.token_stride) + 16 * ((threadIdx.x >> 4) & 3);
            if constexpr (E4M3) sc[b] = scale_off(c, pg, head, slot);
        }
    }
    __device__ __forceinline__ static void load(u32x4_t (&to)[2][J], uint32_t (&exp)[2], const char* from,
                                                const uint8_t* scales, const int64_t (&at)[2], const int64_t (&sc)[2]) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int j = 0; j < J; ++j) to[b][j] = *reinterpret_cast<const u32x4_t*>(from + at[b] + 64 * j);
            if constexpr (E4M3) exp[b] = scales[sc[b]];
        }
    }
    __device__ __forceinline__ void load_k(const Kv& c, int head) { load(k, k_exp, c.k + ES * head * c.head_stride, c.k_scale, at, sc); }
    __device__ __forceinline__ void load_v(const Kv& c, int head) { load(v, v_exp, c.v + ES * head * c.head_stride, c.v_scale, at, sc); }
    __device__ __forceinline__ void store_v(char* vt) const {
        const int col = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                *reinterpret_cast<u32x4_t*>(vt + (16 * b + col) * (2 * D) + 16 * n_chunk<D>(col, q_part(i, g) / 8)) =
                    part(v[b], v_exp[b], i);
    }
};

template <int D, bool E4M3, bool CAREFUL>
__device__ __forceinline__ bool narrow_pass(const AttnArgs& a, const Item& it, int pos, int p_lo, int p_hi, int head,
                                            int w, const u32x4_t (&qf)[D / 32], char* vt, f32x4_t (&acc)[D / 16],
                                            float& m, f32x4_t& l) {
    constexpr int RB = 2 * D, DB = D / 16, KS = D / 32, T = 32;
    typedef NarrowTile<D, E4M3> Tile;
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    const int n = max(0, 2 * it.it1 - 2 * it.it0 - w + 3) >> 2;
    const EveryFourth tile{it.span, 2 * it.it0 + w, 2 * it.it1 - 1};
#pragma unroll
    for (int d = 0; d < DB; ++d) acc[d] = f32x4_t{};
    m = -INFINITY;
    l = f32x4_t{};
    Tile x;
    if (n > 0) {
        x.look_up(a.kv, it, tile(0));
        x.place(a.kv, it, tile(0), head);
        x.look_up(a.kv, it, tile(1));
        x.load_k(a.kv, head);
        x.load_v(a.kv, head);
    }
    for (int i = 0; i < n; ++i) {
        const int t0 = tile(i);
        f32x4_t s[2] = {f32x4_t{}, f32x4_t{}};
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int b = 0; b < 2; ++b) s[b] = mfma16(Tile::part(x.k[b], x.k_exp[b], k), qf[k], s[b]);
        x.store_v(vt);
        if (i + 1 < n) {
            x.place(a.kv, it, tile(i + 1), head);
            x.look_up(a.kv, it, tile(i + 2));
            x.load_k(a.kv, head);
            x.load_v(a.kv, head);
        }
        if (none_sees(a, p_lo, p_hi, t0, t0 + T - 1)) continue;

        const bool masked = !all_see(a, p_lo, p_hi, t0, t0 + T - 1);
        if (masked) hide(a, pos, t0 + 4 * g, [&](auto hidden) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (hidden(16 * b + r)) s[b][r] = -INFINITY;
        });
        float top = s[0][0];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) top = fmaxf(top, s[b][r]);
        const float unit = CAREFUL ? 1.f : a.sl2;  // of m
        if (__ballot(top * unit > m + (CAREFUL ? 0.f : kGrow))) {
            top = fmaxf(top, __shfl_xor(top, 16));
            const float up = fmaxf(m, fmaxf(top, __shfl_xor(top, 32)) * unit);
            const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(CAREFUL ? (m - up) * a.sl2 : m - up);
            m = up;
            l *= f;
#pragma unroll
            for (int d = 0; d < DB; ++d) acc[d] *= f;
        }
        const float off = m == -INFINITY ? 0.f : -m;
        const auto weight = [&](float x) {
            if (CAREFUL) return kCare * __builtin_amdgcn_exp2f((x + off) * a.sl2);
            return __builtin_amdgcn_exp2f(fmaf(x, a.sl2, off));
        };
        uint32_t pw[4], rest[4];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 4; r += 2) {
                const float p0 = weight(s[b][r]), p1 = weight(s[b][r + 1]);
                const uint32_t w = pack_bf16(p0, p1);
                pw[2 * b + r / 2] = w;
                rest[2 * b + r / 2] = pack_bf16(p0 - bf16_lo(w), p1 - bf16_hi(w));
            }
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
            l = add_weights(pw[k], pw[k + 1], l);
            l = add_weights(rest[k], rest[k + 1], l);
        }
        if (CAREFUL && masked) {
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                const uint32_t cur = pw[0], more = rest[0];
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    pw[k] = pw[k + 1];
                    rest[k] = rest[k + 1];
                }
#pragma unroll 1
                for (int x = 0; x < 8; ++x) {
                    const uint32_t both = __shfl(cur, col + 16 * (x >> 1)), add = __shfl(more, col + 16 * (x >> 1));
                    const float p = x & 1 ? bf16_hi(both) + bf16_hi(add) : bf16_lo(both) + bf16_lo(add);
                    const int tok = 16 * (j >> 1) + 4 * (x >> 1) + 2 * (j & 1) + (x & 1);
                    const bool vis = sees(a, pos, t0 + tok);
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int el = 16 * d + 4 * g + e;
                            const float v = v_elem(vt, RB, tok, n_chunk<D>(tok, el >> 3), el & 7);
                            acc[d][e] = vis ? fmaf(p, v, acc[d][e]) : acc[d][e];
                        }
                }
            }
            continue;
        }
        const u32x4_t pf = {pw[0], pw[1], pw[2], pw[3]}, rf = {rest[0], rest[1], rest[2], rest[3]};
        const int r = 4 * g + (col >> 2);
#pragma unroll
        for (int d = 0; d < DB; ++d) {
            const int ch = 2 * d + ((col & 3) >> 1), by = 8 * (col & 1);
            const u32x2_t lo = ds_tr16(vt + r * RB + 16 * n_chunk<D>(r, ch) + by);
            const u32x2_t hi = ds_tr16(vt + (r + 16) * RB + 16 * n_chunk<D>(r, ch) + by);
            const u32x4_t v = {lo[0], lo[1], hi[0], hi[1]};
            acc[d] = mfma16(v, pf, acc[d]);
            acc[d] = mfma16(v, rf, acc[d]);
        }
    }
    if (CAREFUL) m *= a.sl2;
    float bad = fabsf(m) >= kFar && m != -INFINITY ? 1.f : 0.f;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) bad = fmaf(acc[d][e], 0.f, bad);
    return __ballot(bad != 0.f) != 0;
}

// Up to 16 rows (the query heads of a kv head, for a few new tokens): the four
// waves take tiles of 32 tokens in turn, each through LDS of its own, so that
// no barrier stands between the loads, and join their results at the end.
// Every byte of the cache is used once: bound by memory, as far as the tiles in
// flight cover its latency.  One token over each of 64 contexts of 256 to 2048
// (32 kv heads, bf16) takes 146 us, 5.9 TB/s; over each of 32 contexts of 2048
// to 32768 (8 kv heads of 8 query heads, e4m3) 123 us, 5.1 TB/s (136, in an
// earlier form, with the keys through LDS too, which leaves a compute unit two
// workgroups, not three); over a single context of 776 10 us, two launches.  The
// registers are bounded for the workgroups that the plan counts on.
template <int D, bool E4M3>
__global__ __launch_bounds__(256, D == 64 ? 4 : E4M3 ? 3 : 2) void attn_narrow_kernel(AttnArgs a) {
    constexpr int DB = D / 16, KS = D / 32, T = 32;
    __shared__ __align__(16) char lds[4][T * 2 * D];
    __shared__ float s_m[4][16], s_l[4][16];
    const int head = blockIdx.x % a.kv.n_kv_heads, lane = threadIdx.x & 63, w = wave_id();
    const int col = lane & 15, g = lane >> 4;
    Item it;
    if (!load_item(a, blockIdx.x / a.kv.n_kv_heads, AT_NARROW_ROWS, false, it)) return;

    const int row = min(col, it.nrows - 1);
    const int pos = row_pos(a, it, row), p_lo = it.p0, p_hi = row_pos(a, it, it.nrows - 1);
    u32x4_t qf[KS];
    {
        const uint16_t* q = a.q + row_off(a, it, row, head, a.ldq, D);
#pragma unroll
        for (int k = 0; k < KS; ++k)
            qf[k] = *reinterpret_cast<const u32x4_t*>(q + NarrowTile<D, E4M3>::q_part(k, g));
    }
    f32x4_t acc[DB];
    float m;
    f32x4_t sum;
    float unit = 1.f;  // of the sum
    if (narrow_pass<D, E4M3, false>(a, it, pos, p_lo, p_hi, head, w, qf, lds[w], acc, m, sum)) {
        unit = kCare;
        narrow_pass<D, E4M3, true>(a, it, pos, p_lo, p_hi, head, w, qf, lds[w], acc, m, sum);
    }

    // join the waves: each leaves its maximum, sum and [row][D] output in LDS
    float l = sum[0] + __shfl_xor(sum[0], 16);
    l += __shfl_xor(l, 32);
    const float own = reciprocal(l);
    if (g == 0) {
        s_m[w][col] = m;
        s_l[w][col] = l / unit;
    }
    float* mine = reinterpret_cast<float*>(lds[w]);
#pragma unroll
    for (int d = 0; d < DB; ++d) *reinterpret_cast<f32x4_t*>(mine + col * D + 16 * d + 4 * g) = acc[d] * own;
    __syncthreads();
    constexpr int EPT = D / 16;  // elements per thread: 16 threads a row
    const int r = threadIdx.x / 16, e0 = (threadIdx.x % 16) * EPT;
    if (r >= it.nrows) return;
    float top = s_m[0][r], total = 0.f, part[4], o[EPT];
#pragma unroll
    for (int x = 1; x < 4; ++x) top = fmaxf(top, s_m[x][r]);
#pragma unroll
    for (int x = 0; x < 4; ++x) total += part[x] = part_weight(s_m[x][r], s_l[x][r], top);
    const float inv = reciprocal(total);
#pragma unroll
    for (int e = 0; e < EPT; ++e) o[e] = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const float* p = reinterpret_cast<const float*>(lds[x]) + r * D + e0;
#pragma unroll
        for (int e = 0; e < EPT; ++e) o[e] = fmaf(part[x] * inv, p[e], o[e]);
    }
    if (it.nsplits == 1) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row_off(a, it, r, head, a.ldo, D) + e0);
#pragma unroll
        for (int e = 0; e < EPT; e += 2) dst[e / 2] = pack_bf16(o[e], o[e + 1]);
    } else {
        const int64_t pr = head * a.part_rows + it.part + r;
        float* dst = a.part + pr * D + e0;
#pragma unroll
        for (int e = 0; e < EPT; e += 4) *reinterpret_cast<f32x4_t*>(dst + e) = f32x4_t{o[e], o[e + 1], o[e + 2], o[e + 3]};
        if (threadIdx.x % 16 == 0) {
            float* ml = a.part + (int64_t)a.kv.n_kv_heads * a.part_rows * D + 2 * pr;
            ml[0] = top;
            ml[1] = total;
        }
    }
}

// Joins the splits of one row tile, in their order: D/4 lanes a row.  A launch
// of 2 to 5 us, most of it latency: four splits' loads are under way at once.
template <int D>
__global__ __launch_bounds__(256) void attn_merge_kernel(AttnArgs a) {
    constexpr int LPR = D / 4, AHEAD = 4;
    const int head = blockIdx.x % a.kv.n_kv_heads;
    Item it;
    if (!load_item(a, blockIdx.x / a.kv.n_kv_heads, AT_PAIR_ROWS, true, it)) return;
    const int r = it.it0 + threadIdx.x / LPR, e0 = 4 * (threadIdx.x % LPR);
    if (r >= it.it1) return;
    const int64_t first = head * a.part_rows + it.part + r;
    const u32x2_t* ml = reinterpret_cast<const u32x2_t*>(a.part + (int64_t)a.kv.n_kv_heads * a.part_rows * D);
    float top = -INFINITY, sum = 0.f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < it.nsplits; s += AHEAD) {  // AHEAD splits' loads at once
        u32x2_t x[AHEAD];
        f32x4_t p[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t pr = first + (int64_t)min(s + i, it.nsplits - 1) * it.nrows;
            x[i] = ml[pr];
            p[i] = *reinterpret_cast<const f32x4_t*>(a.part + pr * D + e0);
        }
        float up = top;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) up = fmaxf(up, __uint_as_float(x[i][0]));
        float all = part_weight(top, sum, up), part[AHEAD];
        const float old = all;
        top = up;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            part[i] = s + i < it.nsplits ? part_weight(__uint_as_float(x[i][0]), __uint_as_float(x[i][1]), top) : 0.f;
            all += part[i];
        }
        sum = all;
        const float inv = reciprocal(sum);
        o *= old * inv;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (s + i >= it.nsplits) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = fmaf(part[i] * inv, p[i][e], o[e]);
        }
    }
    *reinterpret_cast<u32x2_t*>(a.out + row_off(a, it, r, head, a.ldo, D) + e0) =
        u32x2_t{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
}

// ------------------------------------------------------------------ launchers
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

constexpr int64_t kMaxBlocks = (int64_t)1 << 23;  // of one launch (256 threads each: a grid holds under 2^32)

template <typename A>
hipError_t launch(void (*fn)(A), dim3 grid, dim3 block, hipStream_t s, A& args) {
    void* p[] = {&args};
    return hipLaunchKernel(reinterpret_cast<const void*>(fn), grid, block, p, 0, s);
}

int32_t check_kv(const lora_attn_launch_t* L, const lora_kv_t* c) {
    if (!L || !c || !c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return LORA_EINVAL;
    const lora_attn_info_t& I = L->info;
    const lora_attn_shape_t& s = I.shape;
    if (I.n_seq < 0 || I.n_rows < 0 || I.n_tokens < 0 || (I.n_staged > 0 && !L->meta) || !aligned16(L->meta))
        return LORA_EINVAL;
    if (c->n_pages != s.n_pages || c->page_tokens != s.page_tokens || c->n_kv_heads != s.n_kv_heads ||
        c->head_dim != s.head_dim || c->dtype != s.kv_dtype)
        return LORA_ESHAPE;
    if (s.head_dim != 64 && s.head_dim != 128) return LORA_ESHAPE;
    if (s.n_kv_heads < 1 || s.n_heads < 1 || s.n_heads % s.n_kv_heads || s.page_tokens < 1 ||
        (s.page_tokens & (s.page_tokens - 1)) || s.n_pages < 1)
        return LORA_ESHAPE;
    if (s.window < 0 || s.window > AT_MAX_TOKENS || s.sinks < 0 || s.sinks > AT_MAX_TOKENS) return LORA_EINVAL;
    if (s.kv_dtype != LORA_KV_BF16 && s.kv_dtype != LORA_KV_E4M3) return LORA_EINVAL;
    const int64_t per = s.kv_dtype == LORA_KV_E4M3 ? 16 : 8;
    if (c->page_stride < 0 || c->head_stride < 0 || c->token_stride < 0 || c->page_stride % per ||
        c->head_stride % per || c->token_stride % per)
        return LORA_EINVAL;
    if (s.kv_dtype == LORA_KV_E4M3 && (!c->k_scale || !c->v_scale)) return LORA_EINVAL;
    return LORA_OK;
}
Kv to_kv(const lora_kv_t& c) {
    return Kv{static_cast<const char*>(c.k), static_cast<const char*>(c.v), c.k_scale, c.v_scale, c.page_stride,
              c.head_stride, c.token_stride, c.n_pages, __builtin_ctz((unsigned)c.page_tokens), c.n_kv_heads};
}
bool bad_rows(const void* p, int64_t ld, int64_t d) { return !p || !aligned16(p) || ld < d || ld % 8 != 0; }

}  // namespace

extern "C" int32_t lora_attn_prepare(const lora_attn_shape_t* shape, int32_t n_seq, const int32_t* q_len,
                                     const int32_t* kv_len, const int32_t* block_table, int64_t ld_table,
                                     int32_t* staging, int64_t staging_capacity, void* dev_staging, void* hip_stream,
                                     lora_attn_launch_t* out) {
    if (!out) return LORA_EINVAL;
    out->meta = nullptr;  // info may change with an error, and the calls would take it for the old plan's
    if (!dev_staging || !aligned16(dev_staging)) return LORA_EINVAL;
    const int32_t st = lora_attn_plan(shape, n_seq, q_len, kv_len, block_table, ld_table, staging, staging_capacity,
                                      &out->info);
    if (st != LORA_OK) return st;
    const hipError_t e = hipMemcpyAsync(dev_staging, staging, (size_t)out->info.n_staged * sizeof(int32_t),
                                        hipMemcpyHostToDevice, reinterpret_cast<hipStream_t>(hip_stream));
    if (e != hipSuccess) return LORA_EHIP;
    out->meta = static_cast<const int32_t*>(dev_staging);
    return LORA_OK;
}

extern "C" int32_t lora_kv_write(const lora_attn_launch_t* L, const lora_kv_t* kv, const lora_kv_write_args_t* w,
                                 void* hip_stream) {
    const int32_t st = check_kv(L, kv);
    if (st != LORA_OK) return st;
    if (!w || (w->dtype != LORA_F32 && w->dtype != LORA_BF16)) return LORA_EINVAL;
    const lora_attn_info_t& I = L->info;
    if (I.n_rows == 0) return LORA_OK;
    const int32_t d = I.shape.head_dim, hq = w->q ? I.shape.n_heads : 0, hk = I.shape.n_kv_heads;
    if (bad_rows(w->k, w->ldk, (int64_t)hk * d) || bad_rows(w->v, w->ldv, (int64_t)hk * d)) return LORA_EINVAL;
    if (w->q && (bad_rows(w->q, w->ldq, (int64_t)hq * d) || bad_rows(w->q_out, w->ld_out, (int64_t)hq * d)))
        return LORA_EINVAL;
    if (w->rope_dim < 0 || w->rope_dim > d || w->rope_dim % 16 != 0) return LORA_ESHAPE;
    if ((w->rope_dim > 0) != (w->rope != nullptr) || !aligned16(w->rope)) return LORA_EINVAL;
    if (w->rope && w->rope_len < I.max_kv) return LORA_EINVAL;
    WriteArgs a;
    memset(&a, 0, sizeof(a));
    a.kv = to_kv(*kv);
    a.q = w->q;
    a.k = w->k;
    a.v = w->v;
    a.ldq = w->ldq;
    a.ldk = w->ldk;
    a.ldv = w->ldv;
    a.rope = w->rope;
    a.q_out = w->q_out;
    a.ld_out = w->ld_out;
    a.row_pos = L->meta + I.off_row_pos;
    a.row_slot = L->meta + I.off_row_slot;
    a.n_heads = hq;
    a.n_vec = hq + 2 * hk;
    a.n_rows = I.n_rows;
    a.rope_dim = w->rope_dim;
    a.rope_len = w->rope_len;
    typedef void (*fn_t)(WriteArgs);
    static const fn_t fn[2][2][2] = {
        {{kv_write_kernel<64, false, false>, kv_write_kernel<64, false, true>},
         {kv_write_kernel<64, true, false>, kv_write_kernel<64, true, true>}},
        {{kv_write_kernel<128, false, false>, kv_write_kernel<128, false, true>},
         {kv_write_kernel<128, true, false>, kv_write_kernel<128, true, true>}}};
    const int vpb = 256 / (d / 8);
    const unsigned gy = (unsigned)(I.n_rows < 32768 ? I.n_rows : 32768);
    const dim3 grid((unsigned)((a.n_vec + vpb - 1) / vpb), gy, (unsigned)((I.n_rows + gy - 1) / gy));
    const hipError_t e = launch(fn[d == 128][w->dtype == LORA_F32][kv->dtype == LORA_KV_E4M3], grid, dim3(256),
                                reinterpret_cast<hipStream_t>(hip_stream), a);
    return e == hipSuccess ? LORA_OK : LORA_EHIP;
}

extern "C" int32_t lora_kv_read(const lora_attn_launch_t* L, const lora_kv_t* kv, uint16_t* k_out, uint16_t* v_out,
                                int64_t ld, void* hip_stream) {
    const int32_t st = check_kv(L, kv);
    if (st != LORA_OK) return st;
    const lora_attn_info_t& I = L->info;
    const int32_t d = I.shape.head_dim, hk = I.shape.n_kv_heads;
    if (I.n_tokens == 0) return LORA_OK;
    if (bad_rows(k_out, ld, (int64_t)hk * d) || bad_rows(v_out, ld, (int64_t)hk * d)) return LORA_EINVAL;
    ReadArgs a{to_kv(*kv), k_out, v_out, ld, L->meta + I.off_kv_start, L->meta + I.off_table, I.n_seq, I.n_tokens,
               I.ld_table};
    typedef void (*fn_t)(ReadArgs);
    static const fn_t fn[2][2] = {{kv_read_kernel<64, false>, kv_read_kernel<64, true>},
                                  {kv_read_kernel<128, false>, kv_read_kernel<128, true>}};
    const int64_t vpb = 256 / (d / 8);
    const int64_t blocks = (I.n_tokens + vpb - 1) / vpb * ((hk + kReadHeads - 1) / kReadHeads);
    const hipError_t e = launch(fn[d == 128][kv->dtype == LORA_KV_E4M3],
                                dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), dim3(256),
                                reinterpret_cast<hipStream_t>(hip_stream), a);
    return e == hipSuccess ? LORA_OK : LORA_EHIP;
}

extern "C" int32_t lora_attn(const lora_attn_launch_t* L, const lora_kv_t* kv, const uint16_t* q, int64_t ldq,
                             uint16_t* out, int64_t ldo, float scale, float* workspace, int64_t workspace_floats,
                             void* hip_stream) {
    const int32_t st = check_kv(L, kv);
    if (st != LORA_OK) return st;
    const lora_attn_info_t& I = L->info;
    const int32_t d = I.shape.head_dim, hk = I.shape.n_kv_heads;
    const int64_t width = (int64_t)I.shape.n_heads * d;
    if (I.n_rows == 0) return LORA_OK;
    if (bad_rows(q, ldq, width) || bad_rows(out, ldo, width)) return LORA_EINVAL;
    if (!(scale > 0.f) || !(scale * kLog2e < INFINITY)) return LORA_EINVAL;  // 0 * infinity is no score
    if (I.workspace_floats > 0) {
        if (workspace_floats < I.workspace_floats) return LORA_ECAPACITY;
        if (!workspace || !aligned16(workspace)) return LORA_EINVAL;
    }
    for (const int64_t n : {I.n_work[0], I.n_work[1], I.n_work[2], I.n_merge})
        if (n < 0 || n * hk > kMaxBlocks) return LORA_EINVAL;
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    a.kv = to_kv(*kv);
    a.table = L->meta + I.off_table;
    a.q = q;
    a.out = out;
    a.part = workspace;
    a.ldq = ldq;
    a.ldo = ldo;
    a.part_rows = I.part_rows;
    a.n_seq = I.n_seq;
    a.n_rows = I.n_rows;
    a.max_kv = I.max_kv;
    a.ld_table = I.ld_table;
    a.group = I.shape.n_heads / hk;
    if (a.group > AT_MAX_GROUP) return LORA_ESHAPE;
    a.inv_group = (uint32_t)((((int64_t)1 << 31) + a.group - 1) / a.group);
    a.window = I.shape.window;
    a.sinks = I.shape.sinks;
    a.sl2 = scale * kLog2e;
    const hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
    const bool e4m3 = kv->dtype == LORA_KV_E4M3;
    typedef void (*fn_t)(AttnArgs);
#define AT_FORMS(kernel, d, ...)                                                        \
    {{kernel<d, false, false, ##__VA_ARGS__>, kernel<d, false, true, ##__VA_ARGS__>},   \
     {kernel<d, true, false, ##__VA_ARGS__>, kernel<d, true, true, ##__VA_ARGS__>}}
    static const fn_t wide[2][2][2][2] = {
        {AT_FORMS(attn_wide_kernel, 64, false), AT_FORMS(attn_wide_kernel, 128, false)},
        {AT_FORMS(attn_wide_kernel, 64, true), AT_FORMS(attn_wide_kernel, 128, true)}};
    static const fn_t narrow[2][2] = {{attn_narrow_kernel<64, false>, attn_narrow_kernel<64, true>},
                                      {attn_narrow_kernel<128, false>, attn_narrow_kernel<128, true>}};
#undef AT_FORMS
    // where Places can work with scalar page offsets: a step's rows in one page, 32-bit strides and scale offsets
    const bool uni = kv->page_tokens >= 64 / (d / 8) && kv->token_stride <= INT32_MAX / 64 &&
                     kv->page_stride <= INT32_MAX && (int64_t)kv->n_pages * kv->page_tokens * hk <= UINT32_MAX;
    for (int kind = LORA_ATTN_KINDS - 1; kind >= 0; --kind) {  // the longer items first
        if (I.n_work[kind] == 0) continue;
        a.work = reinterpret_cast<const lora_attn_work_t*>(L->meta + I.off_work[kind]);
        const dim3 grid((unsigned)(I.n_work[kind] * hk)), block(kind == LORA_ATTN_PAIR ? 512 : 256);
        const fn_t fn = kind == LORA_ATTN_NARROW ? narrow[d == 128][e4m3]
                                                 : wide[kind == LORA_ATTN_PAIR][d == 128][e4m3][uni];
        if (launch(fn, grid, block, s, a) != hipSuccess) return LORA_EHIP;
    }
    if (I.n_merge > 0) {
        a.work = reinterpret_cast<const lora_attn_work_t*>(L->meta + I.off_merge);
        const dim3 grid((unsigned)(I.n_merge * hk));
        if (launch(d == 128 ? attn_merge_kernel<128> : attn_merge_kernel<64>, grid, dim3(256), s, a) != hipSuccess)
            return LORA_EHIP;
    }
    return LORA_OK;
}
