// Drives lora_kv_pages_* with exactly sized buffers under the host sanitizers,
// against a plain copy of every sequence's tokens.
#include <stdio.h>

#include <set>
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
    unsigned seed = 11;
    const auto rnd = [&seed](int n) {
        seed = seed * 1664525u + 1013904223u;
        return (int)((seed >> 8) % (unsigned)n);
    };
    for (int t = 0; t < 60; ++t) {
        const int n_pages = 1 + rnd(60), page = 1 << rnd(6), n_seqs = 1 + rnd(9);
        lora_kv_pages_t* P = nullptr;
        CHECK(lora_kv_pages_create(n_pages, page, n_seqs, &P) == LORA_OK);
        std::vector<std::vector<int>> tokens(n_seqs);           // what each sequence holds
        std::vector<int> memory((size_t)n_pages * page, -1);    // what is in the pages
        int next = 0;
        const auto copy = [&](int src, int dst, int len) {
            for (int i = 0; i < len; ++i) memory[(size_t)dst * page + i] = memory[(size_t)src * page + i];
        };
        for (int step = 0; step < 200; ++step) {
            const int what = rnd(10), s = rnd(n_seqs);
            if (what < 5) {
                std::vector<int32_t> seqs, more;
                for (int i = 0; i < n_seqs; ++i)
                    if (rnd(2)) {
                        seqs.push_back(i);
                        more.push_back(rnd(4) ? rnd(3) : rnd(3 * page));
                    }
                const int n = (int)seqs.size();
                std::vector<int32_t> src(n), dst(n), len(n);
                int32_t copies = -1;
                const int32_t st = lora_kv_pages_append(P, n, seqs.data(), more.data(), src.data(), dst.data(), len.data(), &copies);
                CHECK(st == LORA_OK || st == LORA_ECAPACITY);
                if (st != LORA_OK) continue;
                for (int i = 0; i < copies; ++i) copy(src[i], dst[i], len[i]);
                for (int i = 0; i < n; ++i) {
                    int32_t cols, kv;
                    lora_kv_pages_table(P, 1, &seqs[i], 0, nullptr, &kv, &cols);
                    std::vector<int32_t> table(cols);
                    CHECK(lora_kv_pages_table(P, 1, &seqs[i], cols, table.data(), &kv, &cols) == LORA_OK);
                    CHECK(kv == (int)tokens[seqs[i]].size() + more[i]);
                    for (int j = 0; j < more[i]; ++j) {
                        const int at = (int)tokens[seqs[i]].size();
                        tokens[seqs[i]].push_back(next);
                        memory[(size_t)table[at / page] * page + at % page] = next++;
                    }
                }
            } else if (what < 7) {
                std::vector<int32_t> kids;
                for (int i = 0; i < n_seqs; ++i)
                    if (i != s && tokens[i].empty() && rnd(2)) kids.push_back(i);
                CHECK(lora_kv_pages_fork(P, s, (int)kids.size(), kids.data()) == LORA_OK);
                for (const int k : kids) tokens[k] = tokens[s];
            } else if (what == 7) {
                const int keep = rnd((int)tokens[s].size() + 1);
                CHECK(lora_kv_pages_truncate(P, s, keep) == LORA_OK);
                tokens[s].resize(keep);
            } else if (what == 8) {
                const int32_t twice[2] = {s, s};
                CHECK(lora_kv_pages_free(P, 2, twice) == LORA_OK);
                tokens[s].clear();
            } else {
                int32_t moves = -1;
                int32_t st = lora_kv_pages_compact(P, 0, nullptr, nullptr, nullptr, &moves);
                CHECK(st == (moves ? LORA_ECAPACITY : LORA_OK));
                if (moves) {
                    std::vector<int32_t> src(moves), dst(moves), len(moves);
                    CHECK(lora_kv_pages_compact(P, moves, src.data(), dst.data(), len.data(), &moves) == LORA_OK);
                    std::set<int> read(src.begin(), src.end()), written(dst.begin(), dst.end());
                    CHECK((int)read.size() == moves && (int)written.size() == moves);
                    for (const int d : written) CHECK(!read.count(d));
                    for (int i = 0; i < moves; ++i) {
                        CHECK(len[i] >= 1 && len[i] <= page);
                        copy(src[i], dst[i], len[i]);
                    }
                }
                int32_t free_pages, end;
                CHECK(lora_kv_pages_stats(P, &free_pages, nullptr, &end) == LORA_OK && end == n_pages - free_pages);
            }
            std::set<int> used;
            for (int i = 0; i < n_seqs; ++i) {
                int32_t cols, kv;
                const int32_t id = i;
                lora_kv_pages_table(P, 1, &id, 0, nullptr, &kv, &cols);
                std::vector<int32_t> table(cols + 1, 7);
                CHECK(lora_kv_pages_table(P, 1, &id, cols + 1, table.data(), &kv, &cols) == LORA_OK);
                CHECK(kv == (int)tokens[i].size() && table[cols] == 0);
                for (int j = 0; j < kv; ++j) CHECK(memory[(size_t)table[j / page] * page + j % page] == tokens[i][j]);
                used.insert(table.begin(), table.begin() + cols);
            }
            int32_t free_pages;
            CHECK(lora_kv_pages_stats(P, &free_pages, nullptr, nullptr) == LORA_OK);
            CHECK(free_pages == n_pages - (int)used.size());
        }
        lora_kv_pages_destroy(P);
    }
    printf("page manager ok\n");
    return 0;
}
