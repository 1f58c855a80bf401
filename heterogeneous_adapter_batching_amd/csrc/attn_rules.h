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

#endif
