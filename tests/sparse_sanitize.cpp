// Drives lora_sparse_plan with exactly sized buffers under the host sanitizers: what
// it stages lies inside the buffer, and its items cover every row once.
#include <stdio.h>

#include <vector>

#include "hetlora.h"

#define CHECK(x)                                                  \
    do {                                                          \
        if (!(x)) {                                               \
            printf("failed at line %d: %s\n", __LINE__, #x);      \
            return 1;                                             \
        }                                                         \
    } while (0)

int main() {
    unsigned seed = 5;
    const auto rnd = [&seed](int n) {
        seed = seed * 1664525u + 1013904223u;
        return (int)((seed >> 8) % (unsigned)n);
    };
    for (int t = 0; t < 400; ++t) {
        const int hk = 1 + rnd(8), group = rnd(3) ? 1 + rnd(9) : 1 + rnd(40), page = 16 << rnd(4), n = rnd(7);
        const lora_attn_shape_t s = {hk * group, hk, rnd(2) ? 64 : 128, page, 64, rnd(2), 0, 0};
        lora_sparse_shape_t sp = {0, rnd(4), 1 + rnd(3), 0};
        sp.select = sp.first + sp.last + (rnd(3) ? rnd(9) : rnd(400));
        std::vector<int32_t> q(n), kv(n), bounded(n);
        int32_t pages = 0;
        for (int i = 0; i < n; ++i) {
            q[i] = rnd(4) ? rnd(3) : rnd(400);
            kv[i] = rnd(8) ? q[i] + (rnd(6) ? rnd(9000) : rnd(120000)) : rnd(2);
            bounded[i] = rnd(kv[i] + 1);
            const int32_t need = (kv[i] + page - 1) / page;
            pages = need > pages ? need : pages;
        }
        std::vector<int32_t> table((size_t)n * pages);
        for (int32_t& p : table) p = rnd(64);
        const int32_t* b = rnd(2) ? bounded.data() : nullptr;
        lora_attn_info_t attn;
        lora_sparse_info_t info;
        int32_t st = lora_sparse_plan(&s, &sp, n, q.data(), kv.data(), b, table.data(), pages, nullptr, 0, &attn, &info);
        if (st == LORA_EINVAL) continue;  // nothing to stage needs no buffer
        CHECK(st == LORA_ECAPACITY || (st == LORA_OK && attn.n_staged == 0));
        std::vector<int32_t> staging((size_t)attn.n_staged);
        if (attn.n_staged > 0) {
            std::vector<int32_t> less((size_t)attn.n_staged - 1);
            CHECK(lora_sparse_plan(&s, &sp, n, q.data(), kv.data(), b, table.data(), pages, less.data(),
                                   attn.n_staged - 1, &attn, &info) == LORA_ECAPACITY);
        }
        CHECK(lora_sparse_plan(&s, &sp, n, q.data(), kv.data(), b, table.data(), pages, staging.data(), attn.n_staged,
                               &attn, &info) == LORA_OK);
        std::vector<int> seen((size_t)attn.n_rows);
        const auto* items = reinterpret_cast<const lora_sparse_item_t*>(staging.data() + info.off_items);
        for (int i = 0; i < info.n_items; ++i) {
            CHECK(items[i].n >= 1 && items[i].n <= info.item_tokens && items[i].row >= 0 &&
                  items[i].row + items[i].n <= attn.n_rows);
            for (int j = 0; j < items[i].n; ++j) ++seen[(size_t)(items[i].row + j)];
        }
        for (const int x : seen) CHECK(x == 1);
        for (int i = 0; i < info.n_fresh; ++i) CHECK(staging[(size_t)info.off_fresh + i] < 64);
        if (!table.empty() && kv[0] > 0) {
            table[0] = 64;
            CHECK(lora_sparse_plan(&s, &sp, n, q.data(), kv.data(), b, table.data(), pages, staging.data(), attn.n_staged,
                                   &attn, &info) == LORA_EPAGE);
            table[0] = 0;
            bounded[0] = kv[0] + 1;
            CHECK(lora_sparse_plan(&s, &sp, n, q.data(), kv.data(), bounded.data(), table.data(), pages, staging.data(),
                                   attn.n_staged, &attn, &info) == LORA_EINVAL);
        }
    }
    printf("sparse planner ok\n");
    return 0;
}
