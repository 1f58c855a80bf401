// Drives lora_attn_plan over its whole ranges with exactly sized buffers under the
// host sanitizers.  Every batch here is valid, so the planner has to take it.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <vector>

#include "hetlora.h"

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
                rows += w[i].it0 == 0 ? w[i].nrows : 0;
            }
        }
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
