// What the kernels on the paged cache share: element types, where a token lies,
// and the checks and launches of their C entry points.
#ifndef HETLORA_KV_DEVICE_H
#define HETLORA_KV_DEVICE_H

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
typedef short s16x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int32_t s32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// Two fp32 -> packed bf16, round to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const bf16x2_t p = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

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

// Where chunk c (16 bytes) of a row lies in LDS, rows of 2 D bytes: the 16 lanes that
// read one chunk of 16 rows hit all banks once.
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c) {
    return c ^ (D == 128 ? row & 15 : (row >> 1) & 7);
}
// Everything that the wave has written to LDS is there for its other lanes.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ------------------------------------------------------------------ launchers
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

constexpr int64_t kMaxBlocks = (int64_t)1 << 23;  // of one launch (256 threads each: a grid holds under 2^32)

template <typename A>
hipError_t launch(void (*fn)(A), dim3 grid, dim3 block, hipStream_t s, A& args) {
    void* p[] = {&args};
    return hipLaunchKernel(reinterpret_cast<const void*>(fn), grid, block, p, 0, s);
}

inline int32_t check_kv(const lora_attn_launch_t* L, const lora_kv_t* c) {
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
// A plan that no cache is given with, and its sparse part.
inline int32_t check_sparse(const lora_sparse_launch_t& L) {
    const lora_attn_info_t& I = L.attn.info;
    const lora_attn_shape_t& s = I.shape;
    const lora_sparse_info_t& S = L.info;
    if (I.n_seq < 0 || I.n_rows < 0 || I.n_tokens < 0 || (I.n_staged > 0 && !L.attn.meta) || !aligned16(L.attn.meta))
        return LORA_EINVAL;
    if ((s.head_dim != 64 && s.head_dim != 128) || s.n_kv_heads < 1 || s.n_heads < 1 || s.n_heads % s.n_kv_heads ||
        s.n_heads / s.n_kv_heads > AT_MAX_GROUP || s.page_tokens < SP_MIN_PAGE ||
        (s.page_tokens & (s.page_tokens - 1)) || s.n_pages < 1)
        return LORA_ESHAPE;
    if (s.window != 0 || s.sinks != 0 || S.shape.first < 0 || S.shape.last < 1 || S.shape.select > AT_MAX_TOKENS ||
        S.shape.select < (int64_t)S.shape.first + S.shape.last)
        return LORA_EINVAL;
    if (S.n_items < 0 || S.n_work < 0 || S.n_merge < 0 || S.n_fresh < 0 || S.max_scored < 0 || S.item_tokens < 1)
        return LORA_EINVAL;
    return LORA_OK;
}
inline Kv to_kv(const lora_kv_t& c) {
    return Kv{static_cast<const char*>(c.k), static_cast<const char*>(c.v), c.k_scale, c.v_scale, c.page_stride,
              c.head_stride, c.token_stride, c.n_pages, __builtin_ctz((unsigned)c.page_tokens), c.n_kv_heads};
}
inline bool bad_rows(const void* p, int64_t ld, int64_t d) { return !p || !aligned16(p) || ld < d || ld % 8 != 0; }

}  // namespace

#endif
