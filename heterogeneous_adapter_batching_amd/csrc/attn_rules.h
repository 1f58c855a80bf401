// Rules of the attention plan that the host planner and the kernels share:
// how a range of query positions maps to tiles of cached tokens.  Plain
// C/C++ with no HIP dependency.
#ifndef HETLORA_ATTN_RULES_H
#define HETLORA_ATTN_RULES_H

#include <stdint.h>

#include "../../include/hetlora.h"

#ifndef AT_FN
#define AT_FN static inline
#endif

#define AT_TILE 64          // cached tokens of one tile
// Most new and cached tokens of a sequence: positions are in [-AT_MAX_TOKENS,
// AT_MAX_TOKENS), so a longer window hides nothing and more sinks are all there
// are.  The plan takes the smaller, and a position minus a window fits 32 bits.
#define AT_MAX_TOKENS (1 << 30)
// query rows of one item of the kernels
#define AT_NARROW_ROWS 16
#define AT_WIDE_ROWS 128
#define AT_PAIR_ROWS 256
// most query heads of a kv head: the kernels divide numbers below this and 256 by it
#define AT_MAX_GROUP 4096
// rows of one merge entry: 256 threads, four elements each
#define AT_MERGE_ROWS(head_dim) (1024 / (head_dim))

// Tiles that queries at positions p_lo .. p_hi may see, as a list: the first
// `sinks` tiles 0 .. sinks-1, then `first` .. `end`-1.
struct AtSpan {
    int32_t sinks, first, end;
};

AT_FN int32_t at_min(int32_t a, int32_t b) { return a < b ? a : b; }
AT_FN int32_t at_max(int32_t a, int32_t b) { return a > b ? a : b; }

AT_FN struct AtSpan at_span(int32_t p_lo, int32_t p_hi, int32_t window, int32_t sinks) {
    struct AtSpan s = {0, 0, 0};
    if (p_hi < 0) return s;
    s.end = p_hi / AT_TILE + 1;
    if (window > 0) {
        s.first = at_max(0, p_lo - window + 1) / AT_TILE;
        s.sinks = at_min((int32_t)(((int64_t)sinks + AT_TILE - 1) / AT_TILE), s.first);
    }
    return s;
}
AT_FN int32_t at_span_tiles(struct AtSpan s) { return s.sinks + s.end - s.first; }
AT_FN int32_t at_span_tile(struct AtSpan s, int32_t i) { return i < s.sinks ? i : s.first + (i - s.sinks); }

// An item (or merge entry) of at most max_rows rows lies inside the batch and the
// workspace.  last_tok = (lead + nrows - 1) / group.
AT_FN int at_inside(const lora_attn_work_t* w, int32_t n_seq, int32_t n_rows, int32_t max_kv, int32_t group,
                    int32_t max_rows, int64_t part_rows, int32_t last_tok, int merge) {
    if (w->seq < 0 || w->seq >= n_seq || w->n_new < 0 || w->kv < 0 || w->kv > max_kv || w->q0 < 0 ||
        w->q0 + (int64_t)w->n_new > n_rows)
        return 0;
    if (w->nrows < 1 || w->nrows > max_rows || w->tok0 < 0 || w->lead < 0 || w->lead >= group ||
        w->tok0 + (int64_t)last_tok >= w->n_new)
        return 0;
    if (w->nsplits < 1) return 0;
    if ((merge || w->nsplits > 1) &&
        (w->part < 0 || w->part + (int64_t)w->nrows * (merge ? w->nsplits : 1) > part_rows))
        return 0;
    return 1;
}

// ------------------------------------------------------------------ sparse attention
#define SP_MIN_PAGE 16       // fewest tokens of a page: under that its bounds are as much as its keys
#define SP_EXP 100           // exponents of bounds are within +-SP_EXP
// Keys (scores) that a selecting workgroup of several tokens holds in LDS at most, tiles
// of 16 rows (query heads of its tokens) that it scores one after another at most, and
// its waves, each of which chooses for a token.  More tokens than waves only as 2, 4 or 8
// times as many, and with few keys: us of 2048 tokens, 8 kv heads of 2 query heads, over
//              8 tokens   16   24
//   282 pages      36.5 28.5 46.0
//   560            53.1 69.9
// and of 512 tokens, 32 kv heads of their own, over
//              8 tokens   16   32
//   70 pages      25.4 18.1 15.0
//   250           34.4 24.7 29.7
//   500           50.2 35.8
// 2048 tokens, 64/8 heads, over 282 pages: two tiles at most 67.7, four 54.7.
#define SP_LDS_KEYS 12288
#define SP_ROW_TILES 4
#define SP_WAVES 8
#define SP_FEW_KEYS 4096
// Of a single token's keys, which one workgroup scores where it holds them; more are
// scored by many workgroups, into memory, and chosen from by another launch.  us in
// LDS and through memory, one token of each sequence, 8 kv heads of 8 query heads:
//   pages         500       1000       2000       4000       8000
//   1 sequence   7.5/11.9   9.9/12.7  14.5/13.4  28.6/14.9  50.7/16.7
//   16           8.0/12.5  11.3/14.3  18.3/20.3  37.4/30.6  73.5/55.7
//   64          18.8/23.5  29.7/34.2  53.2/59.4
// (One sequence alone would gain from some 1900 pages on; the rule is the same for any
// number of them.)  The batch's longest context decides for all of it: 64/8 heads, pages of
// 16, 512 tokens over 16512 take 60 us, one over 131072 19, both in one batch 312, with
// one token to an item; 63 single tokens over 8192 20, one over 40000 14, all 64 32.
#define SP_ONE_KEYS 2048
#define SP_SLAB_KEYS (1 << 24)  // keys in memory at once

AT_FN int sp_in_lds(int32_t max_scored, int32_t item_tokens) {
    return (int64_t)max_scored * item_tokens <= (item_tokens > 1 ? SP_LDS_KEYS : SP_ONE_KEYS);
}
// items of one launch, where the keys of each (of one token, all heads') go through memory
AT_FN int64_t sp_slab(int64_t per_item, int64_t n_items) {
    const int64_t fit = SP_SLAB_KEYS / per_item;
    return fit < 1 ? 1 : fit < n_items ? fit : n_items;
}

#endif
