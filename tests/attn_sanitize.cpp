// Drives lora_attn_plan with exactly sized buffers under the host sanitizers.
#include <stdio.h>
#include <stdlib.h>

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
    unsigned seed = 7;
    const auto rnd = [&seed](int n) {
        seed = seed * 1664525u + 1013904223u;
        return (int)((seed >> 8) % (unsigned)n);
    };
    for (int t = 0; t < 400; ++t) {
        const int hk = 1 + rnd(8), group = 1 + rnd(9), page = 1 << rnd(8), n = rnd(7);
        lora_attn_shape_t s = {hk * group, hk, rnd(2) ? 64 : 128, page, 64, rnd(2), rnd(3) * rnd(300), rnd(3) * rnd(90)};
        std::vector<int32_t> q(n), kv(n);
        int32_t pages = 0;
        for (int i = 0; i < n; ++i) {
            q[i] = rnd(4) ? rnd(3) : rnd(400);
            kv[i] = rnd(8) ? q[i] + rnd(3000) : rnd(2);
            const int32_t need = (kv[i] + page - 1) / page;
            pages = need > pages ? need : pages;
        }
        std::vector<int32_t> table((size_t)n * pages);
        for (int32_t& p : table) p = rnd(64);
        lora_attn_info_t info;
        int32_t st = lora_attn_plan(&s, n, q.data(), kv.data(), table.data(), pages, nullptr, 0, &info);
        if (st == LORA_EINVAL) continue;  // nothing to stage needs no buffer
        CHECK(st == LORA_ECAPACITY || (st == LORA_OK && info.n_staged == 0));
        std::vector<int32_t> staging((size_t)info.n_staged);
        CHECK(lora_attn_plan(&s, n, q.data(), kv.data(), table.data(), pages, staging.data(), info.n_staged, &info) ==
              LORA_OK);
        if (!table.empty() && kv[0] > 0) {
            table[0] = 64;
            CHECK(lora_attn_plan(&s, n, q.data(), kv.data(), table.data(), pages, staging.data(), info.n_staged,
                                 &info) == LORA_EPAGE);
        }
    }
    printf("attention planner ok\n");
    return 0;
}
