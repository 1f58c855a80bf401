// Drives lora_attn_plan over its whole ranges with exactly sized buffers under the
// host sanitizers, and the kernels' own check of its items.  Every batch here is
// valid, so the planner has to take it.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <vector>

#include "attn_rules.h"

#define CHECK(x)                                                  \
    do {                                                          \
        if (!(x)) {                                               \
            printf("failed at line %d: %s\n", __LINE__, #x);      \
            return 1;                                             \
        }                                                         \
    } while (0)

static unsigned seed = 11;
static int rnd(int n) {
    seed = seed * 1664525u + 1013904223u;
    return (int)((seed >> 8) % (unsigned)n);
}
// 0, small, or up to the largest of its type
static int32_t wide() {
    switch (rnd(4)) {
        case 0: return 0;
        case 1: return 1 + rnd(600);
        case 2: return INT32_MAX - rnd(3);
        default: return (1 << 30) - 1 + rnd(3);
    }
}

static bool inside(const lora_attn_work_t& w, const lora_attn_info_t& info, int max_rows, bool merge) {
    const int32_t group = info.shape.n_heads / info.shape.n_kv_heads;
    return at_inside(&w, info.n_seq, info.n_rows, info.max_kv, group, max_rows, info.part_rows,
                     (int32_t)(((int64_t)w.lead + w.nrows - 1) / group), merge) != 0;
}
// Numbers that would lead a kernel out of its buffers are not inside.
static int broken_items(const lora_attn_work_t& good, const lora_attn_info_t& info, int max_rows, bool merge) {
    CHECK(inside(good, info, max_rows, merge));
    const int32_t last = INT32_MAX;
    const struct {
        int32_t lora_attn_work_t::*field;
        int32_t value;
    } bad[] = {{&lora_attn_work_t::seq, -1},       {&lora_attn_work_t::seq, info.n_seq},
               {&lora_attn_work_t::nrows, 0},      {&lora_attn_work_t::nrows, max_rows + 1},
               {&lora_attn_work_t::nsplits, 0},    {&lora_attn_work_t::nsplits, -1},
               {&lora_attn_work_t::q0, -1},        {&lora_attn_work_t::q0, last},
               {&lora_attn_work_t::n_new, 0},      {&lora_attn_work_t::n_new, last},
               {&lora_attn_work_t::kv, -1},        {&lora_attn_work_t::kv, last},
               {&lora_attn_work_t::tok0, -1},      {&lora_attn_work_t::tok0, last},
               {&lora_attn_work_t::lead, -1},      {&lora_attn_work_t::lead, info.shape.n_heads}};
    for (const auto& b : bad) {
        lora_attn_work_t w = good;
        w.*b.field = b.value;
        CHECK(!inside(w, info, max_rows, merge));
    }
    lora_attn_work_t w = good;
    w.nsplits = merge ? good.nsplits : 2;
    for (const int64_t part : {(int64_t)-1, info.part_rows, (int64_t)last}) {
        w.part = (int32_t)std::min<int64_t>(part, last);
        CHECK(!inside(w, info, max_rows, merge));
    }
    w.part = -1;
    w.nsplits = 1;
    CHECK(inside(w, info, max_rows, merge) == !merge);  // a merge reads parts however many it says
    return 0;
}

int main() {
    int splits = 0, before = 0, far = 0;
    for (int t = 0; t < 600; ++t) {
        const int hk = 1 + rnd(8), group = 1 + rnd(9), page = 1 << rnd(11), n = rnd(7);
        const lora_attn_shape_t s = {hk * group, hk, rnd(2) ? 64 : 128, page, 64, rnd(2), wide(), wide()};
        std::vector<int32_t> q(n), kv(n);
        int32_t pages = 0;
        for (int i = 0; i < n; ++i) {
            q[i] = rnd(3) ? rnd(3) : rnd(400);
            kv[i] = rnd(3) == 0 ? rnd(q[i] + 1) : q[i] + rnd(rnd(3) ? 300 : 20000);  // a third have rows before token 0
            before += q[i] > kv[i];
            const int32_t need = (kv[i] + page - 1) / page;
            pages = std::max(pages, need);
        }
        far += s.window > 1 << 30 && before > 0;
        std::vector<int32_t> table((size_t)n * pages);
        for (int32_t& p : table) p = rnd(64);
        lora_attn_info_t info;
        CHECK(lora_attn_plan(&s, n, q.data(), kv.data(), table.data(), pages, nullptr, 0, &info) == LORA_ECAPACITY);
        CHECK(info.n_staged > n);
        std::vector<int32_t> staging((size_t)info.n_staged);
        CHECK(lora_attn_plan(&s, n, q.data(), kv.data(), table.data(), pages, staging.data(), info.n_staged - 1, &info) ==
              LORA_ECAPACITY);
        CHECK(lora_attn_plan(&s, n, q.data(), kv.data(), table.data(), pages, staging.data(), info.n_staged, &info) ==
              LORA_OK);
        splits += info.n_merge > 0;
        int64_t rows = 0, want = 0;
        for (int i = 0; i < n; ++i) want += (int64_t)q[i] * group;
        for (int kind = 0; kind < LORA_ATTN_KINDS; ++kind) {
            const lora_attn_work_t* w = reinterpret_cast<const lora_attn_work_t*>(staging.data() + info.off_work[kind]);
            for (int i = 0; i < info.n_work[kind]; ++i) {
                CHECK(0 <= w[i].it0 && w[i].it0 <= w[i].it1);
                const int most[] = {AT_NARROW_ROWS, AT_WIDE_ROWS, AT_PAIR_ROWS};
                if (broken_items(w[i], info, most[kind], false)) return 1;
                rows += w[i].it0 == 0 ? w[i].nrows : 0;
            }
        }
        for (int i = 0; i < info.n_merge; ++i)
            if (broken_items(reinterpret_cast<const lora_attn_work_t*>(staging.data() + info.off_merge)[i], info,
                             AT_PAIR_ROWS, true))
                return 1;
        CHECK(rows >= want);  // a row tile's first split, and empty ones
        if (n > 0 && kv[0] > 0) {
            table[0] = 64;
            CHECK(lora_attn_plan(&s, n, q.data(), kv.data(), table.data(), pages, staging.data(), info.n_staged,
                                 &info) == LORA_EPAGE);
        }
    }
    CHECK(splits > 100 && before > 100 && far > 50);
    printf("attention planner ok over its ranges\n");
    return 0;
}
