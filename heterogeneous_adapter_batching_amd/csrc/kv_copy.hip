// gfx950 kernel that copies pages of a paged cache, and its C entry point.
#include <stddef.h>

#include <algorithm>
#include <functional>
#include <new>
#include <vector>

#include "kv_device.h"

namespace {

// One cache's tensors.
struct CopyCache {
    char *k, *v;
    uint8_t *k_scale, *v_scale;
    int8_t* codes;  // bounds, or none
    uint8_t* exps;
};
struct CopyPair {
    int32_t from, to, tokens;
};
// Caches and pairs travel in the launch's arguments: nothing is staged, and the
// lists are free again when the call returns.  Copies within caches have one entry
// to a cache, others the source's and, CACHES / 2 on, the destination's.  A launch
// with the few pairs of a decode step has short arguments
// (one pair in one cache: 4.1 us for 4.5, and 19 for 25 when it is waited for).
template <int CACHES, int PAIRS>
struct CopyArgs {
    static constexpr int kCaches = CACHES, kPairs = PAIRS;
    int64_t from_page, from_head, from_token, to_page, to_head, to_token;  // strides in bytes
    int32_t n_heads, page_shift, token_blocks, bound_bytes, to_cache;
    CopyCache cache[CACHES];
    CopyPair pair[PAIRS];
};
typedef CopyArgs<8, 16> CopyFew;
typedef CopyArgs<32, 192> CopyMany;
static_assert(sizeof(CopyMany) <= 4096, "a kernel's arguments are at most 4 KiB");

// VPR lanes take a token of a head, 16 bytes of its key and of its value each, and a
// workgroup 256 / VPR tokens: of one head, or where a page holds fewer of several
// heads side by side.  Bound by memory: 64 forks inside pages of 16 (8 kv heads,
// bf16, 32 layers: 132 MB moved) take 24.7 us, 5.4 TB/s; 700 whole e4m3 pages of 64
// of 4 layers, with scales and bounds (751 MB), 154 us, 4.9 TB/s in four launches.
// Small workgroups, since all of a launch's copies are under way at once anyway: two
// and four such steps to a workgroup take 26.5 and 27.9 us (fork).  Stores go past
// the caches (without: 32.7 and 174); loads, of pages that may have been written a step
// before, from kCopyPast bytes of a call on.  us without and with that, 8 caches of 8
// heads of 128, whole pages, the same ones again and again, which the caches hold as far
// as they can, and three sets of pages in turn:
//   bf16, pages of 16   129 MB 41/50 51/52   160 50/63 64/64   200 65/78 81/79   300 106/119 123/121   500 209/205 208/205
//   e4m3,          64   130    40/47 46/48   161 49/60 60/60   201 60/73 76/74   302 102/115 118/115   503 196/192 198/193
// (The gain is small: of pages that were all written right before, a call of 200 to 300 MB
// loses more than others gain.)
constexpr int64_t kCopyPast = 200000000;
template <int VPR, bool SCALES, bool PAST, typename Args>
__global__ __launch_bounds__(256) void kv_copy_kernel(Args a) {
    constexpr int ROWS = 256 / VPR;
    const CopyCache &c = a.cache[blockIdx.z], &t = a.cache[blockIdx.z + a.to_cache];
    const CopyPair p = a.pair[blockIdx.y];
    const int shift = min(a.page_shift, __builtin_ctz(ROWS));  // tokens of a workgroup
    const int row = threadIdx.x / VPR, col = threadIdx.x % VPR;
    const int token = ((int)(blockIdx.x % a.token_blocks) << shift) + (row & ((1 << shift) - 1));
    const int head = (int)(blockIdx.x / a.token_blocks) * (ROWS >> shift) + (row >> shift);
    if (token < p.tokens && head < a.n_heads) {
        const int64_t at = p.from * a.from_page + head * a.from_head + token * a.from_token + 16 * col;
        const int64_t to = p.to * a.to_page + head * a.to_head + token * a.to_token + 16 * col;
        const u32x4_t *kp = reinterpret_cast<const u32x4_t*>(c.k + at), *vp = reinterpret_cast<const u32x4_t*>(c.v + at);
        const u32x4_t k = PAST ? __builtin_nontemporal_load(kp) : *kp, v = PAST ? __builtin_nontemporal_load(vp) : *vp;
        if (SCALES && col == 0) {
            const int64_t s = (((int64_t)p.from * a.n_heads + head) << a.page_shift) + token;
            const int64_t d = (((int64_t)p.to * a.n_heads + head) << a.page_shift) + token;
            t.k_scale[d] = c.k_scale[s];
            t.v_scale[d] = c.v_scale[s];
        }
        __builtin_nontemporal_store(k, reinterpret_cast<u32x4_t*>(t.k + to));
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(t.v + to));
    }
    // bounds of a whole page, all heads': one workgroup of the page
    if (c.codes && blockIdx.x == 0 && p.tokens >> a.page_shift) {
        const int64_t bytes = (int64_t)a.n_heads * a.bound_bytes;
        for (int64_t i = 16 * threadIdx.x; i < bytes; i += 16 * 256)
            *reinterpret_cast<u32x4_t*>(t.codes + p.to * bytes + i) =
                *reinterpret_cast<const u32x4_t*>(c.codes + p.from * bytes + i);
        for (int h = threadIdx.x; h < a.n_heads; h += 256)
            t.exps[(int64_t)p.to * a.n_heads + h] = c.exps[(int64_t)p.from * a.n_heads + h];
    }
}

int32_t check_cache(const lora_kv_t& c, const lora_kv_t& like) {
    if (!c.k || !c.v || !aligned16(c.k) || !aligned16(c.v) || c.n_pages < 1 || c.n_kv_heads < 1) return LORA_EINVAL;
    if (c.dtype != LORA_KV_BF16 && c.dtype != LORA_KV_E4M3) return LORA_EINVAL;
    if ((c.head_dim != 64 && c.head_dim != 128) || c.n_kv_heads > 65535) return LORA_ESHAPE;
    if (c.page_tokens < 1 || c.page_tokens > 1024 || (c.page_tokens & (c.page_tokens - 1)) != 0) return LORA_ESHAPE;
    if (c.dtype != like.dtype || c.head_dim != like.head_dim || c.n_kv_heads != like.n_kv_heads ||
        c.page_tokens != like.page_tokens || c.n_pages != like.n_pages)
        return LORA_ESHAPE;
    const int64_t per = c.dtype == LORA_KV_E4M3 ? 16 : 8;
    if (c.page_stride < 0 || c.head_stride < 0 || c.token_stride < 0 || c.page_stride % per || c.head_stride % per ||
        c.token_stride % per)
        return LORA_EINVAL;
    if (c.dtype == LORA_KV_E4M3 && (!c.k_scale || !c.v_scale)) return LORA_EINVAL;
    return LORA_OK;
}
int32_t check_bounds(const lora_kv_bounds_t& b, const lora_kv_t& c) {
    if (!b.codes || !b.exps || !aligned16(b.codes)) return LORA_EINVAL;
    if (b.n_pages != c.n_pages || b.n_kv_heads != c.n_kv_heads || b.head_dim != c.head_dim) return LORA_ESHAPE;
    return LORA_OK;
}
CopyCache side(const lora_kv_t& c, const lora_kv_bounds_t* b) {
    return CopyCache{static_cast<char*>(c.k), static_cast<char*>(c.v), c.k_scale, c.v_scale, b ? b->codes : nullptr,
                     b ? b->exps : nullptr};
}
bool same_strides(const lora_kv_t& a, const lora_kv_t& b) {
    return a.page_stride == b.page_stride && a.head_stride == b.head_stride && a.token_stride == b.token_stride;
}

// A tensor that is written, and where from; strides of the pages' tensors, and of
// the others a number for their kind.
struct Written {
    const void *to, *from;
    int32_t cache;
    int64_t page_stride, head_stride, token_stride;
    bool operator<(const Written& o) const { return std::less<const void*>()(to, o.to); }
    bool alike(const Written& o) const {
        return from == o.from && page_stride == o.page_stride && head_stride == o.head_stride && token_stride == o.token_stride;
    }
};
// Memory that is read and also written: of keys, values or scales, of bounds by
// their own copy, and of bounds by another cache's.
struct Shared {
    bool pages, bounds, others_bounds;
};

// No memory is written twice, but by copies that write the same: of keys and values
// that are one tensor on both sides, and within caches (which may be listed twice)
// wherever the layouts are the same.  Scales and exponents count where there is
// something to copy.
int32_t check_tensors(bool within, bool any, int32_t n, const lora_kv_t* from, const lora_kv_t* to,
                      const lora_kv_bounds_t* from_bounds, const lora_kv_bounds_t* to_bounds, Shared& shared) {
    shared = {within, false, false};
    if (within && std::all_of(from, from + n, [&](const lora_kv_t& c) { return same_strides(c, from[0]); })) return LORA_OK;
    try {
        std::vector<Written> written;
        for (int32_t i = 0; i < n; ++i) {
            const auto add = [&](const void* t, const void* f, int64_t page, int64_t head, int64_t token) {
                if (t) written.push_back({t, f, i, page, head, token});
            };
            add(to[i].k, from[i].k, to[i].page_stride, to[i].head_stride, to[i].token_stride);
            add(to[i].v, from[i].v, to[i].page_stride, to[i].head_stride, to[i].token_stride);
            if (within) continue;
            if (to_bounds) add(to_bounds[i].codes, from_bounds[i].codes, -1, 0, 0);
            if (!any) continue;
            if (to[i].dtype == LORA_KV_E4M3) {
                add(to[i].k_scale, from[i].k_scale, -2, 0, 0);
                add(to[i].v_scale, from[i].v_scale, -2, 0, 0);
            }
            if (to_bounds) add(to_bounds[i].exps, from_bounds[i].exps, -3, 0, 0);
        }
        std::sort(written.begin(), written.end());
        for (size_t i = 1; i < written.size(); ++i) {
            const Written &x = written[i - 1], &y = written[i];
            if (x.to == y.to && !((within || x.cache == y.cache) && x.alike(y))) return LORA_EINVAL;
        }
        if (within) return LORA_OK;
        const auto find = [&](const void* p) {  // what writes it, or none
            const auto at = std::lower_bound(written.begin(), written.end(), Written{p, nullptr, 0, 0, 0, 0});
            return p && at != written.end() && at->to == p ? &*at : nullptr;
        };
        for (int32_t i = 0; i < n; ++i) {
            for (const void* p : {(const void*)from[i].k, (const void*)from[i].v, (const void*)from[i].k_scale,
                                  (const void*)from[i].v_scale})
                shared.pages |= find(p) != nullptr;
            for (const void* p : {from[i].k, from[i].v}) {  // in one layout: others' pages overlap otherwise
                const Written* by = find(p);
                if (by && by->page_stride >= 0 && (by->page_stride != from[i].page_stride ||
                    by->head_stride != from[i].head_stride || by->token_stride != from[i].token_stride))
                    return LORA_EINVAL;
            }
            if (!from_bounds) continue;
            for (const void* p : {(const void*)from_bounds[i].codes, (const void*)from_bounds[i].exps}) {
                const Written* by = find(p);
                shared.bounds |= by && by->cache == i;
                shared.others_bounds |= by && by->cache != i;
            }
        }
    } catch (const std::bad_alloc&) {
        return LORA_ENOMEM;
    }
    return LORA_OK;
}

// Every page that is written is written once, and none is read that is also
// written where source and destination share memory.  (Bounds go with whole pages
// only, and may stay where they are.)
int32_t check_pairs(int32_t n, const int32_t* from, const int32_t* to, const int32_t* tokens, int32_t from_pages,
                    int32_t to_pages, int32_t page_tokens, const Shared& shared) {
    for (int32_t i = 0; i < n; ++i) {
        if (from[i] < 0 || from[i] >= from_pages || to[i] < 0 || to[i] >= to_pages) return LORA_EPAGE;
        if (tokens && (tokens[i] < 0 || tokens[i] > page_tokens)) return LORA_EINVAL;
    }
    const bool bounds = shared.bounds || shared.others_bounds;
    if (n < 2 && !(n == 1 && (shared.pages || bounds))) return LORA_OK;
    try {
        std::vector<int32_t> written(to, to + n);
        std::sort(written.begin(), written.end());
        if (std::adjacent_find(written.begin(), written.end()) != written.end()) return LORA_EINVAL;
        if (shared.pages) {
            for (int32_t i = 0; i < n; ++i)
                if (std::binary_search(written.begin(), written.end(), from[i])) return LORA_EINVAL;
        } else if (bounds) {
            const auto whole = [&](int32_t i) { return !tokens || tokens[i] == page_tokens; };
            written.clear();
            for (int32_t i = 0; i < n; ++i)
                if (whole(i)) written.push_back(to[i]);
            std::sort(written.begin(), written.end());
            for (int32_t i = 0; i < n; ++i)
                if (whole(i) && (shared.others_bounds || from[i] != to[i]) &&
                    std::binary_search(written.begin(), written.end(), from[i]))
                    return LORA_EINVAL;
        }
    } catch (const std::bad_alloc&) {
        return LORA_ENOMEM;
    }
    return LORA_OK;
}

// Every argument has been checked; within caches (not `across`) `to` is `from`.
template <typename Args>
int32_t copy_pages(bool across, int32_t n_caches, const lora_kv_t* from, const lora_kv_t* to, const lora_kv_bounds_t* from_bounds,
                   const lora_kv_bounds_t* to_bounds, int32_t n_pairs, const int32_t* from_page, const int32_t* to_page,
                   const int32_t* tokens, void* hip_stream) {
    const lora_kv_t& c = from[0];
    const bool e4m3 = c.dtype == LORA_KV_E4M3;
    const int es = e4m3 ? 1 : 2, vpr = c.head_dim * es / 16, rows = 256 / vpr;
    const int32_t block = std::min(c.page_tokens, rows);  // tokens of a workgroup
    const int32_t token_blocks = c.page_tokens / block, heads = rows / block;
    Args a;
    memset(&a, 0, offsetof(Args, cache));
    a.n_heads = c.n_kv_heads;
    a.page_shift = __builtin_ctz((unsigned)c.page_tokens);
    a.token_blocks = token_blocks;
    a.bound_bytes = 2 * c.head_dim;
    const int32_t most = across ? Args::kCaches / 2 : Args::kCaches;  // caches of a launch
    a.to_cache = across ? most : 0;
    typedef void (*fn_t)(Args);
    static const fn_t fns[2][2][2] = {{{kv_copy_kernel<8, false, false, Args>, kv_copy_kernel<8, false, true, Args>},
                                       {kv_copy_kernel<16, false, false, Args>, kv_copy_kernel<16, false, true, Args>}},
                                      {{kv_copy_kernel<4, true, false, Args>, kv_copy_kernel<4, true, true, Args>},
                                       {kv_copy_kernel<8, true, false, Args>, kv_copy_kernel<8, true, true, Args>}}};
    int64_t bytes = 0;
    for (int32_t j = 0; j < n_pairs; ++j) bytes += tokens ? tokens[j] : c.page_tokens;
    bytes *= (int64_t)2 * n_caches * c.n_kv_heads * c.head_dim * es;
    const fn_t fn = fns[e4m3][c.head_dim == 128][bytes >= kCopyPast];
    const unsigned gx = (unsigned)(token_blocks * ((c.n_kv_heads + heads - 1) / heads));
    for (int32_t i = 0; i < n_caches;) {
        int32_t n = 0;  // caches of one launch: those on end with the same strides
        for (; i + n < n_caches && n < most && same_strides(from[i], from[i + n]) && same_strides(to[i], to[i + n]); ++n) {
            a.cache[n] = side(from[i + n], from_bounds ? from_bounds + i + n : nullptr);
            if (across) a.cache[n + most] = side(to[i + n], to_bounds ? to_bounds + i + n : nullptr);
        }
        a.from_page = from[i].page_stride * es;
        a.from_head = from[i].head_stride * es;
        a.from_token = from[i].token_stride * es;
        a.to_page = to[i].page_stride * es;
        a.to_head = to[i].head_stride * es;
        a.to_token = to[i].token_stride * es;
        for (int32_t j = 0; j < n_pairs;) {
            int32_t m = 0;
            for (; j < n_pairs && m < Args::kPairs; ++j) {
                const int32_t count = tokens ? tokens[j] : c.page_tokens;
                if (count > 0) a.pair[m++] = CopyPair{from_page[j], to_page[j], count};
            }
            if (m > 0 && launch(fn, dim3(gx, (unsigned)m, (unsigned)n), dim3(256),
                                reinterpret_cast<hipStream_t>(hip_stream), a) != hipSuccess)
                return LORA_EHIP;
        }
        i += n;
    }
    return LORA_OK;
}

}  // namespace

extern "C" int32_t lora_kv_copy(int32_t n_caches, const lora_kv_t* from, const lora_kv_t* to,
                                const lora_kv_bounds_t* from_bounds, const lora_kv_bounds_t* to_bounds, int32_t n_pairs,
                                const int32_t* from_page, const int32_t* to_page, const int32_t* tokens,
                                void* hip_stream) {
    if (n_caches < 1 || n_pairs < 0 || !from || (n_pairs > 0 && (!from_page || !to_page))) return LORA_EINVAL;
    if (!to && to_bounds) return LORA_EINVAL;
    if (to && (from_bounds != nullptr) != (to_bounds != nullptr)) return LORA_EINVAL;
    const lora_kv_t* dst = to ? to : from;
    const lora_kv_bounds_t* dst_bounds = to ? to_bounds : from_bounds;
    for (int32_t i = 0; i < n_caches; ++i) {
        int32_t st = check_cache(from[i], from[0]);
        if (st == LORA_OK && to) st = check_cache(to[i], to[0]);
        if (st == LORA_OK && from_bounds) st = check_bounds(from_bounds[i], from[i]);
        if (st == LORA_OK && dst_bounds) st = check_bounds(dst_bounds[i], dst[i]);
        if (st != LORA_OK) return st;
    }
    const lora_kv_t& c = from[0];
    if (dst->dtype != c.dtype || dst->head_dim != c.head_dim || dst->n_kv_heads != c.n_kv_heads ||
        dst->page_tokens != c.page_tokens)
        return LORA_ESHAPE;
    Shared shared;
    int32_t st = check_tensors(!to, n_pairs > 0, n_caches, from, dst, from_bounds, dst_bounds, shared);
    if (st == LORA_OK) st = check_pairs(n_pairs, from_page, to_page, tokens, c.n_pages, dst->n_pages, c.page_tokens, shared);
    if (st != LORA_OK) return st;

    const int32_t most = to ? CopyFew::kCaches / 2 : CopyFew::kCaches;
    const auto copy = n_pairs <= CopyFew::kPairs && n_caches <= most ? copy_pages<CopyFew> : copy_pages<CopyMany>;
    return copy(to != nullptr, n_caches, from, dst, from_bounds, dst_bounds, n_pairs, from_page, to_page, tokens, hip_stream);
}
