// Host planner of the attention over a paged cache: batch metadata and work
// items.  Plain C++17 with no HIP dependency, like host.cpp.
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "../../include/hetlora.h"
#include "attn_rules.h"

namespace {

constexpr int64_t kUnits = 256;  // compute units
// Workgroups of each kernel that are counted to a compute unit: what its registers
// leave room for.  (The bf16 wide form for 64-wide heads leaves room for three;
// counting them changes nothing that was measured, 56.6 us for 16 prompts of up to
// 2048 tokens either way.)
int64_t resident(int kind, const lora_attn_shape_t& s) {
    if (kind != LORA_ATTN_NARROW) return kind == LORA_ATTN_WIDE ? 2 : 1;
    return s.head_dim == 64 ? 4 : s.kv_dtype == LORA_KV_E4M3 ? 3 : 2;
}
// Tiles of one split, for `tiles` tiles of all heads together: what fills the
// chip's places once where that is kFullTiles at least, else up to kFullTiles
// with one workgroup to a compute unit, and never under kMinTiles.  A split's
// partial result and its part of the merge cost as much as a few tiles do: one
// token over each of 8 windows of 4096 (8 kv heads) takes 31.9 us in splits of 8
// tiles and 30.7 in splits of 16 or 32; over a single context of 776, where most
// compute units are idle, 14.8 us whole, 11.9 in splits of 8 and 10.2 in 4.
// One token over each of 32 e4m3 contexts of up to 32768 takes 123 us on three
// places to a unit, 141 on two, 129 on four.
constexpr int64_t kMinTiles = 4, kFullTiles = 16;
int64_t tiles_per_split(int64_t tiles, int64_t places) {
    const int64_t once = (tiles + places - 1) / places, spread = (tiles + kUnits - 1) / kUnits;
    return once >= kFullTiles ? once : std::max(kMinTiles, std::min(kFullTiles, spread));
}
// Fewest tiles of a pair item.  It has one workgroup to a compute unit, whose
// start nothing else covers, and 256 rows end later than 128 on a causal mask;
// its halves alternate without a gap once it runs.  us, pair and wide:
//   head_dim, cache                  64 bf16  64 e4m3  128 bf16  128 e4m3
//   16 prompts of up to 2048 tokens   87/57   105/68    125/104   149/106
//   2 x 512 tokens over 6000         119/134  151/152   191/213   208/244
//   the same in pages of 2           127/148  167/166   201/239   245/266
//   2 x 512 tokens over 16000        292/336  369/381   471/561   570/613
//   2 x 1024 tokens over 33k            -        -     1904/2300     -
// (Where a chunk straddles the limit both kernels run, one after the other: over
// 1800 tokens, 29 to 41 tiles, that takes 7 to 16 us more than either alone.)
constexpr int32_t kPairTiles = 32;

// Items of a selection, of all kv heads together, that are wanted at least.
constexpr int64_t kSelectItems = 2 * kUnits;

struct Tile {  // one row tile of one sequence before it is split
    lora_attn_work_t work;
    int32_t tiles;
};

int32_t check_shape(const lora_attn_shape_t& s) {
    if (s.n_heads < 1 || s.n_kv_heads < 1 || s.n_pages < 1 || s.window < 0 || s.sinks < 0) return LORA_EINVAL;
    if (s.kv_dtype != LORA_KV_BF16 && s.kv_dtype != LORA_KV_E4M3) return LORA_EINVAL;
    if ((s.head_dim != 64 && s.head_dim != 128) || s.n_heads % s.n_kv_heads != 0 || s.n_kv_heads > 65535 ||
        s.n_heads / s.n_kv_heads > AT_MAX_GROUP)
        return LORA_ESHAPE;
    if (s.page_tokens < 1 || s.page_tokens > 1024 || (s.page_tokens & (s.page_tokens - 1)) != 0) return LORA_ESHAPE;
    if ((int64_t)s.n_pages * s.page_tokens > INT32_MAX) return LORA_EINVAL;
    return LORA_OK;
}

// Cuts the row tiles of one kernel into splits and appends items and merges.
void split(const std::vector<Tile>& tiles, int64_t places, const lora_attn_shape_t& s,
           std::vector<lora_attn_work_t>& work, std::vector<lora_attn_work_t>& merge, int64_t& part_rows) {
    int64_t total = 0;
    for (const Tile& t : tiles) total += t.tiles;
    const int64_t share = tiles_per_split(total * s.n_kv_heads, places);
    for (const Tile& t : tiles) {
        const int32_t n = (int32_t)std::max<int64_t>(1, (t.tiles + share / 2) / share);
        lora_attn_work_t w = t.work;
        w.nsplits = n;
        const int64_t first = part_rows;
        for (int32_t i = 0; i < n; ++i) {
            w.it0 = (int32_t)((int64_t)t.tiles * i / n);
            w.it1 = (int32_t)((int64_t)t.tiles * (i + 1) / n);
            w.part = n > 1 ? (int32_t)part_rows : -1;
            work.push_back(w);
            if (n > 1) part_rows += w.nrows;
        }
        if (n == 1) continue;
        const int32_t step = AT_MERGE_ROWS(s.head_dim);
        w.part = (int32_t)first;
        for (int32_t r = 0; r < w.nrows; r += step) {
            w.it0 = r;
            w.it1 = std::min(r + step, w.nrows);
            merge.push_back(w);
        }
    }
    // longest first, so that the last workgroups to start are short
    std::stable_sort(work.begin(), work.end(), [](const lora_attn_work_t& a, const lora_attn_work_t& b) {
        return a.it1 - a.it0 > b.it1 - b.it0;
    });
}

int32_t plan_impl(const lora_attn_shape_t& s, int32_t n_seq, const int32_t* q_len, const int32_t* kv_len,
                  const int32_t* table, int64_t ld_table, int32_t* staging, int64_t capacity,
                  lora_attn_info_t* info) {
    const int32_t group = s.n_heads / s.n_kv_heads;
    int64_t n_rows = 0, n_tokens = 0;
    int32_t pages = 0, max_kv = 0;
    for (int32_t b = 0; b < n_seq; ++b) {
        if (q_len[b] < 0 || kv_len[b] < 0 || kv_len[b] > AT_MAX_TOKENS || q_len[b] > AT_MAX_TOKENS) return LORA_EINVAL;
        n_rows += q_len[b];
        n_tokens += kv_len[b];
        if ((int64_t)q_len[b] * group > INT32_MAX / 2) return LORA_EINVAL;
        const int32_t need = (kv_len[b] + s.page_tokens - 1) / s.page_tokens;
        if (need > ld_table) return LORA_EINVAL;
        pages = std::max(pages, need);
        max_kv = std::max(max_kv, kv_len[b]);
    }
    if (n_rows * group > INT32_MAX / 2 || n_tokens > INT32_MAX) return LORA_EINVAL;
    if (pages > 0 && table == nullptr) return LORA_EINVAL;
    for (int32_t b = 0; b < n_seq; ++b) {
        const int32_t need = (kv_len[b] + s.page_tokens - 1) / s.page_tokens;
        const int32_t* row = table + (need ? b * ld_table : 0);
        for (int32_t i = 0; i < need; ++i)
            if (row[i] < 0 || row[i] >= s.n_pages) return LORA_EPAGE;
    }

    std::vector<Tile> tiles[LORA_ATTN_KINDS];
    int32_t q0 = 0;
    for (int32_t b = 0; b < n_seq; ++b) {
        const int32_t rows = q_len[b] * group, p0 = kv_len[b] - q_len[b];
        for (int32_t r = 0, n = 0; r < rows; r += n) {
            const int32_t left = rows - r;
            const auto tiles_of = [&](int32_t m) {
                return at_span_tiles(at_span(p0 + r / group, p0 + (r + m - 1) / group, s.window, s.sinks));
            };
            // the last rows of a chunk stay with the others: a launch of their
            // own would follow the wide one and take longer than they do in it
            int kind = rows <= AT_NARROW_ROWS ? LORA_ATTN_NARROW : LORA_ATTN_WIDE;
            n = std::min(left, (int32_t)AT_WIDE_ROWS);
            if (left > AT_WIDE_ROWS && tiles_of(n) >= kPairTiles) {
                kind = LORA_ATTN_PAIR;
                n = std::min(left, (int32_t)AT_PAIR_ROWS);
            }
            tiles[kind].push_back({{b, r, n, 0, 0, 1, -1, q0, q_len[b], kv_len[b], r / group, r % group}, tiles_of(n)});
        }
        q0 += q_len[b];
    }
    std::vector<lora_attn_work_t> work[LORA_ATTN_KINDS], merge;
    int64_t part_rows = 0;
    for (int kind = 0; kind < LORA_ATTN_KINDS; ++kind)
        split(tiles[kind], kUnits * resident(kind, s), s, work[kind], merge, part_rows);

    if (part_rows > INT32_MAX) return LORA_EINVAL;
    constexpr int64_t wi = sizeof(lora_attn_work_t) / sizeof(int32_t);
    lora_attn_info_t out;
    memset(&out, 0, sizeof(out));
    out.shape = s;
    out.n_seq = n_seq;
    out.n_rows = (int32_t)n_rows;
    out.n_tokens = (int32_t)n_tokens;
    out.max_kv = max_kv;
    out.ld_table = pages;
    out.n_merge = (int32_t)merge.size();
    out.part_rows = part_rows;
    out.workspace_floats = part_rows * s.n_kv_heads * (s.head_dim + 2);
    int64_t off = 0;
    const auto place = [&off](int64_t n) {  // parts start at multiples of four elements (16 bytes)
        const int64_t at = off;
        off += (n + 3) / 4 * 4;
        return at;
    };
    for (int kind = 0; kind < LORA_ATTN_KINDS; ++kind) {
        out.n_work[kind] = (int32_t)work[kind].size();
        out.off_work[kind] = place(wi * out.n_work[kind]);
    }
    out.off_merge = place(wi * out.n_merge);
    out.off_kv_start = place(n_seq + 1);
    out.off_row_pos = place(n_rows);
    out.off_row_slot = place(n_rows);
    out.off_table = place((int64_t)n_seq * pages);
    out.n_staged = off;
    *info = out;
    if (off > capacity) return LORA_ECAPACITY;
    if (off > 0 && staging == nullptr) return LORA_EINVAL;

    const auto put = [staging](int64_t at, const std::vector<lora_attn_work_t>& v) {
        if (!v.empty()) memcpy(staging + at, v.data(), v.size() * sizeof(lora_attn_work_t));
    };
    for (int kind = 0; kind < LORA_ATTN_KINDS; ++kind) put(out.off_work[kind], work[kind]);
    put(out.off_merge, merge);
    int32_t* kv_start = staging + out.off_kv_start;
    int32_t row = 0, token = 0;
    for (int32_t b = 0; b < n_seq; ++b) {
        kv_start[b] = token;
        const int32_t* src = table + (pages ? b * ld_table : 0);
        for (int32_t i = 0; i < q_len[b]; ++i, ++row) {
            const int32_t p = kv_len[b] - q_len[b] + i;
            staging[out.off_row_pos + row] = p;
            staging[out.off_row_slot + row] =
                p < 0 ? -1 : src[p / s.page_tokens] * s.page_tokens + p % s.page_tokens;
        }
        token += kv_len[b];
        const int32_t need = (kv_len[b] + s.page_tokens - 1) / s.page_tokens;
        int32_t* dst = staging + out.off_table + (int64_t)b * pages;
        if (need) memcpy(dst, src, sizeof(int32_t) * (size_t)need);
        std::fill(dst + need, dst + pages, 0);
    }
    kv_start[n_seq] = token;
    return LORA_OK;
}

// The sparse part behind a plan of the same batch.  Every new token is a sequence
// of its own to the attention: the tokens of its pages on end, the own page's up
// to itself, so that nothing is left to mask; its page table is what the
// selection writes.
int32_t sparse_impl(const lora_attn_shape_t& s, const lora_sparse_shape_t& sp, int32_t n_seq, const int32_t* q_len,
                    const int32_t* kv_len, const int32_t* bounded, const int32_t* table, int64_t ld_table,
                    int32_t* staging, int64_t capacity, lora_attn_info_t* attn, lora_sparse_info_t* info) {
    const int32_t group = s.n_heads / s.n_kv_heads, page = s.page_tokens;
    for (int32_t b = 0; b < n_seq && bounded; ++b)
        if (bounded[b] < 0 || bounded[b] > kv_len[b]) return LORA_EINVAL;
    lora_sparse_info_t out;
    memset(&out, 0, sizeof(out));
    out.shape = sp;
    int32_t pad = 1;  // rows of a token in a tile of 16
    while (pad < 16 && pad < group) pad *= 2;
    int64_t rows = 0;
    const int64_t always = (int64_t)sp.first + sp.last;
    for (int32_t b = 0; b < n_seq; ++b)
        if (q_len[b] > 0 && kv_len[b] > 0) {
            const int32_t pages = (kv_len[b] - 1) / page + 1;
            if (pages > sp.select) out.max_scored = std::max(out.max_scored, (int32_t)(pages - always));
            rows += q_len[b];
        }
    // Tokens of an item: their rows fill the tiles that are scored one after another,
    // their scores fit LDS, and there are items enough to fill the chip.
    const int64_t spread = rows * s.n_kv_heads / kSelectItems;
    out.item_tokens = (int32_t)std::max<int64_t>(
        1, std::min({(int64_t)(16 * SP_ROW_TILES / pad), (int64_t)(SP_LDS_KEYS / std::max(1, out.max_scored)), spread}));
    if (out.item_tokens > SP_WAVES) {  // as many to each wave, and two workgroups to a compute unit
        int32_t n = SP_WAVES;
        while (2 * n <= out.item_tokens && 2 * n * (int64_t)out.max_scored <= (n == SP_WAVES ? 2 : 1) * SP_FEW_KEYS) n *= 2;
        out.item_tokens = n;
    }

    std::vector<lora_sparse_item_t> items;
    std::vector<Tile> tiles;
    std::vector<int32_t> fresh;
    int32_t row = 0;
    for (int32_t b = 0; b < n_seq; ++b) {
        const int32_t p0 = kv_len[b] - q_len[b];
        for (int32_t i = 0; i < q_len[b]; i += out.item_tokens)
            items.push_back({b, row + i, std::min(out.item_tokens, q_len[b] - i), p0 + i});
        for (int32_t i = 0; i < q_len[b]; ++i, ++row) {
            const int32_t p = p0 + i;
            const int32_t kv = p < 0 ? 0 : (std::min(p / page + 1, sp.select) - 1) * page + p % page + 1;
            for (int32_t r = 0; r < group; r += AT_NARROW_ROWS) {
                const int32_t n = std::min(group - r, (int32_t)AT_NARROW_ROWS);
                tiles.push_back({{row, r, n, 0, 0, 1, -1, row, 1, kv, 0, r}, (kv + AT_TILE - 1) / AT_TILE});
            }
        }
        const int32_t from = bounded ? bounded[b] : std::max(0, p0);
        for (int32_t i = from / page; i < kv_len[b] / page; ++i) fresh.push_back(table[b * ld_table + i]);
    }
    std::vector<lora_attn_work_t> work, merge;
    int64_t part_rows = 0;
    split(tiles, kUnits * resident(LORA_ATTN_NARROW, s), s, work, merge, part_rows);
    if (part_rows > INT32_MAX || items.size() > INT32_MAX || work.size() > INT32_MAX || merge.size() > INT32_MAX ||
        fresh.size() > INT32_MAX)
        return LORA_EINVAL;
    out.n_items = (int32_t)items.size();
    out.n_work = (int32_t)work.size();
    out.n_merge = (int32_t)merge.size();
    out.n_fresh = (int32_t)fresh.size();
    out.part_rows = part_rows;
    int64_t floats = part_rows * s.n_kv_heads * (s.head_dim + 2);
    if (!sp_in_lds(out.max_scored, out.item_tokens)) {
        const int64_t per = (int64_t)out.max_scored * s.n_kv_heads;
        floats = std::max(floats, per * sp_slab(per, out.n_items));
    }
    int64_t off = attn->n_staged;
    const auto place = [&off](int64_t n) {
        const int64_t at = off;
        off += (n + 3) / 4 * 4;
        return at;
    };
    constexpr int64_t wi = sizeof(lora_attn_work_t) / sizeof(int32_t), si = sizeof(lora_sparse_item_t) / sizeof(int32_t);
    out.off_items = place(si * out.n_items);
    out.off_work = place(wi * out.n_work);
    out.off_merge = place(wi * out.n_merge);
    out.off_fresh = place(out.n_fresh);
    attn->n_staged = off;
    attn->workspace_floats = std::max(attn->workspace_floats, floats);
    *info = out;
    if (off > capacity) return LORA_ECAPACITY;
    if (off > 0 && staging == nullptr) return LORA_EINVAL;
    if (!items.empty()) memcpy(staging + out.off_items, items.data(), items.size() * sizeof(lora_sparse_item_t));
    if (!work.empty()) memcpy(staging + out.off_work, work.data(), work.size() * sizeof(lora_attn_work_t));
    if (!merge.empty()) memcpy(staging + out.off_merge, merge.data(), merge.size() * sizeof(lora_attn_work_t));
    if (!fresh.empty()) memcpy(staging + out.off_fresh, fresh.data(), fresh.size() * sizeof(int32_t));
    return LORA_OK;
}

}  // namespace

extern "C" int32_t lora_attn_plan(const lora_attn_shape_t* shape, int32_t n_seq, const int32_t* q_len,
                                  const int32_t* kv_len, const int32_t* block_table, int64_t ld_table,
                                  int32_t* staging, int64_t staging_capacity, lora_attn_info_t* info) {
    if (!shape || !info || n_seq < 0 || ld_table < 0 || staging_capacity < 0 || (n_seq > 0 && (!q_len || !kv_len)))
        return LORA_EINVAL;
    const int32_t st = check_shape(*shape);
    if (st != LORA_OK) return st;
    lora_attn_shape_t s = *shape;
    s.window = std::min(s.window, AT_MAX_TOKENS);
    s.sinks = std::min(s.sinks, AT_MAX_TOKENS);
    try {
        return plan_impl(s, n_seq, q_len, kv_len, block_table, ld_table, staging, staging_capacity, info);
    } catch (const std::bad_alloc&) {
        return LORA_ENOMEM;
    }
}

extern "C" int32_t lora_sparse_plan(const lora_attn_shape_t* shape, const lora_sparse_shape_t* sparse, int32_t n_seq,
                                    const int32_t* q_len, const int32_t* kv_len, const int32_t* bounded,
                                    const int32_t* block_table, int64_t ld_table, int32_t* staging,
                                    int64_t staging_capacity, lora_attn_info_t* attn, lora_sparse_info_t* info) {
    if (!shape || !sparse || !attn || !info) return LORA_EINVAL;
    if (shape->window != 0 || shape->sinks != 0) return LORA_EINVAL;
    if (sparse->first < 0 || sparse->last < 1 || sparse->select > AT_MAX_TOKENS ||
        sparse->select < (int64_t)sparse->first + sparse->last)
        return LORA_EINVAL;
    const int32_t st = lora_attn_plan(shape, n_seq, q_len, kv_len, block_table, ld_table, staging, staging_capacity, attn);
    if (st != LORA_OK && st != LORA_ECAPACITY) return st;
    if (shape->page_tokens < SP_MIN_PAGE) return LORA_ESHAPE;
    try {
        return sparse_impl(*shape, *sparse, n_seq, q_len, kv_len, bounded, block_table, ld_table, staging,
                           staging_capacity, attn, info);
    } catch (const std::bad_alloc&) {
        return LORA_ENOMEM;
    }
}
