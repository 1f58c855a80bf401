// Manager of a paged cache's pages (host state only): which pages hold which
// sequence's tokens, how many sequences share a page, and which are free.  It
// says what has to be copied (lora_kv_copy) and moves nothing itself.  Plain
// C++17 with no HIP dependency, like pool.cpp.
#include <stdint.h>

#include <algorithm>
#include <new>
#include <vector>

#include "../../include/hetlora.h"
#include "attn_rules.h"

struct lora_kv_pages {
    int32_t n_pages = 0, page_tokens = 0;
    struct Seq {
        std::vector<int32_t> pages;
        int32_t tokens = 0;
    };
    std::vector<Seq> seqs;
    std::vector<int32_t> users;       // sequences that hold each page
    std::vector<int32_t> free_pages;  // stack; room for all pages, so that a push takes no memory
    std::vector<uint8_t> listed;      // scratch of append and fork: sequences seen so far

    int32_t pages_for(int64_t tokens) const { return (int32_t)((tokens + page_tokens - 1) / page_tokens); }
    void drop(int32_t page) {
        if (--users[(size_t)page] == 0) free_pages.push_back(page);
    }
    int32_t take() {
        const int32_t page = free_pages.back();
        free_pages.pop_back();
        users[(size_t)page] = 1;
        return page;
    }
    bool has(int32_t seq) const { return seq >= 0 && seq < (int32_t)seqs.size(); }
    // The last page is shared and the next token goes into it.
    bool splits(const Seq& s, int32_t more) const {
        return more > 0 && s.tokens % page_tokens != 0 && users[(size_t)s.pages.back()] > 1;
    }
};

namespace {

// Memory runs out in a vector at most: everything is reserved before state changes.
template <typename F>
int32_t guarded(F f) {
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return LORA_ENOMEM;
    }
}

int32_t append(lora_kv_pages& P, int32_t n, const int32_t* seqs, const int32_t* tokens, int32_t* src, int32_t* dst,
               int32_t* len, int32_t* n_copies) {
    int32_t st = LORA_OK;
    for (int32_t i = 0; i < n && st == LORA_OK; ++i) {
        if (!P.has(seqs[i]) || tokens[i] < 0 || P.listed[(size_t)seqs[i]] ||
            (int64_t)P.seqs[(size_t)seqs[i]].tokens + tokens[i] > AT_MAX_TOKENS)
            st = LORA_EINVAL;
        else
            P.listed[(size_t)seqs[i]] = 1;
    }
    for (int32_t i = 0; i < n; ++i)
        if (P.has(seqs[i])) P.listed[(size_t)seqs[i]] = 0;
    if (st != LORA_OK) return st;

    // Splits one after the other: the last holder of a page keeps it.
    int64_t need = 0;
    std::vector<int32_t> left;  // (page) of splits, once each
    left.reserve((size_t)n);
    for (int32_t i = 0; i < n; ++i) {
        const lora_kv_pages::Seq& s = P.seqs[(size_t)seqs[i]];
        const int32_t pages = P.pages_for((int64_t)s.tokens + tokens[i]);
        need += pages - (int32_t)s.pages.size();
        if (P.splits(s, tokens[i])) left.push_back(s.pages.back());
    }
    std::sort(left.begin(), left.end());
    for (size_t i = 0; i < left.size();) {
        size_t end = i;
        while (end < left.size() && left[end] == left[i]) ++end;
        need += std::min<int64_t>((int64_t)(end - i), P.users[(size_t)left[i]] - 1);
        i = end;
    }
    if (need > (int64_t)P.free_pages.size()) return LORA_ECAPACITY;
    for (int32_t i = 0; i < n; ++i) {
        lora_kv_pages::Seq& s = P.seqs[(size_t)seqs[i]];
        s.pages.reserve((size_t)P.pages_for((int64_t)s.tokens + tokens[i]));
    }

    int32_t copies = 0;
    for (int32_t i = 0; i < n; ++i) {
        lora_kv_pages::Seq& s = P.seqs[(size_t)seqs[i]];
        if (P.splits(s, tokens[i])) {
            const int32_t page = s.pages.back();
            src[copies] = page;
            dst[copies] = P.take();
            len[copies] = s.tokens % P.page_tokens;
            s.pages.back() = dst[copies++];
            P.drop(page);
        }
        s.tokens += tokens[i];
        while ((int32_t)s.pages.size() < P.pages_for(s.tokens)) s.pages.push_back(P.take());
    }
    *n_copies = copies;
    return LORA_OK;
}

void truncate(lora_kv_pages& P, lora_kv_pages::Seq& s, int32_t tokens) {
    while ((int32_t)s.pages.size() > P.pages_for(tokens)) {
        P.drop(s.pages.back());
        s.pages.pop_back();
    }
    s.tokens = tokens;
}

int32_t compact(lora_kv_pages& P, int32_t capacity, int32_t* src, int32_t* dst, int32_t* len, int32_t* n_moves) {
    const int32_t used = P.n_pages - (int32_t)P.free_pages.size();
    std::vector<int32_t> to((size_t)P.n_pages), filled((size_t)P.n_pages, 0);
    int32_t moves = 0;
    for (int32_t p = used; p < P.n_pages; ++p) moves += P.users[(size_t)p] > 0;
    *n_moves = moves;
    if (moves > capacity) return LORA_ECAPACITY;
    for (const lora_kv_pages::Seq& s : P.seqs)
        for (size_t i = 0; i < s.pages.size(); ++i) {
            const int64_t in = std::min<int64_t>(P.page_tokens, s.tokens - (int64_t)i * P.page_tokens);
            int32_t& f = filled[(size_t)s.pages[i]];
            f = std::max(f, (int32_t)in);
        }
    int32_t hole = 0, m = 0;
    for (int32_t p = 0; p < P.n_pages; ++p) {
        to[(size_t)p] = p;
        if (p < used || P.users[(size_t)p] == 0) continue;
        while (P.users[(size_t)hole] > 0) ++hole;  // below `used`: as many holes there as pages in use from there on
        to[(size_t)p] = hole;
        src[m] = p;
        dst[m] = hole;
        len[m++] = filled[(size_t)p];
        P.users[(size_t)hole] = P.users[(size_t)p];
        P.users[(size_t)p] = 0;
    }
    for (lora_kv_pages::Seq& s : P.seqs)
        for (int32_t& page : s.pages) page = to[(size_t)page];
    P.free_pages.clear();
    for (int32_t p = P.n_pages - 1; p >= used; --p) P.free_pages.push_back(p);
    return LORA_OK;
}

}  // namespace

extern "C" int32_t lora_kv_pages_create(int32_t n_pages, int32_t page_tokens, int32_t n_seqs, lora_kv_pages_t** out) {
    if (!out || n_pages < 1 || n_seqs < 1) return LORA_EINVAL;
    if (page_tokens < 1 || page_tokens > 1024 || (page_tokens & (page_tokens - 1)) != 0) return LORA_ESHAPE;
    if ((int64_t)n_pages * page_tokens > INT32_MAX) return LORA_EINVAL;
    lora_kv_pages* P = new (std::nothrow) lora_kv_pages;
    if (!P) return LORA_ENOMEM;
    const int32_t st = guarded([&] {
        P->n_pages = n_pages;
        P->page_tokens = page_tokens;
        P->seqs.resize((size_t)n_seqs);
        P->listed.assign((size_t)n_seqs, 0);
        P->users.assign((size_t)n_pages, 0);
        P->free_pages.resize((size_t)n_pages);
        for (int32_t i = 0; i < n_pages; ++i) P->free_pages[(size_t)i] = n_pages - 1 - i;  // page 0 goes first
        return LORA_OK;
    });
    if (st != LORA_OK) {
        delete P;
        return st;
    }
    *out = P;
    return LORA_OK;
}

extern "C" int32_t lora_kv_pages_destroy(lora_kv_pages_t* P) {
    delete P;
    return LORA_OK;
}

extern "C" int32_t lora_kv_pages_append(lora_kv_pages_t* P, int32_t n, const int32_t* seqs, const int32_t* tokens,
                                        int32_t* src, int32_t* dst, int32_t* len, int32_t* n_copies) {
    if (!P || n < 0 || !n_copies || (n > 0 && (!seqs || !tokens || !src || !dst || !len))) return LORA_EINVAL;
    *n_copies = 0;
    return guarded([&] { return append(*P, n, seqs, tokens, src, dst, len, n_copies); });
}

extern "C" int32_t lora_kv_pages_fork(lora_kv_pages_t* P, int32_t parent, int32_t n, const int32_t* children) {
    if (!P || n < 0 || (n > 0 && !children) || !P->has(parent)) return LORA_EINVAL;
    bool good = true;
    for (int32_t i = 0; i < n && good; ++i) {
        good = P->has(children[i]) && children[i] != parent && P->seqs[(size_t)children[i]].tokens == 0 &&
               !P->listed[(size_t)children[i]];
        if (good) P->listed[(size_t)children[i]] = 1;
    }
    for (int32_t i = 0; i < n; ++i)
        if (P->has(children[i])) P->listed[(size_t)children[i]] = 0;
    if (!good) return LORA_EINVAL;
    return guarded([&] {
        const lora_kv_pages::Seq& from = P->seqs[(size_t)parent];
        for (int32_t i = 0; i < n; ++i) P->seqs[(size_t)children[i]].pages.reserve(from.pages.size());
        for (int32_t i = 0; i < n; ++i) {
            lora_kv_pages::Seq& s = P->seqs[(size_t)children[i]];
            s.pages.assign(from.pages.begin(), from.pages.end());
            s.tokens = from.tokens;
            for (const int32_t page : s.pages) ++P->users[(size_t)page];
        }
        return LORA_OK;
    });
}

extern "C" int32_t lora_kv_pages_truncate(lora_kv_pages_t* P, int32_t seq, int32_t tokens) {
    if (!P || !P->has(seq) || tokens < 0 || tokens > P->seqs[(size_t)seq].tokens) return LORA_EINVAL;
    truncate(*P, P->seqs[(size_t)seq], tokens);
    return LORA_OK;
}

extern "C" int32_t lora_kv_pages_free(lora_kv_pages_t* P, int32_t n, const int32_t* seqs) {
    if (!P || n < 0 || (n > 0 && !seqs)) return LORA_EINVAL;
    for (int32_t i = 0; i < n; ++i)
        if (!P->has(seqs[i])) return LORA_EINVAL;
    for (int32_t i = 0; i < n; ++i) truncate(*P, P->seqs[(size_t)seqs[i]], 0);
    return LORA_OK;
}

extern "C" int32_t lora_kv_pages_compact(lora_kv_pages_t* P, int32_t capacity, int32_t* src, int32_t* dst, int32_t* len,
                                         int32_t* n_moves) {
    if (!P || capacity < 0 || !n_moves || (capacity > 0 && (!src || !dst || !len))) return LORA_EINVAL;
    return guarded([&] { return compact(*P, capacity, src, dst, len, n_moves); });
}

extern "C" int32_t lora_kv_pages_table(const lora_kv_pages_t* P, int32_t n, const int32_t* seqs, int64_t ld_table,
                                       int32_t* table, int32_t* kv_len, int32_t* n_columns) {
    if (!P || n < 0 || ld_table < 0 || !n_columns || (n > 0 && (!seqs || !kv_len || (ld_table > 0 && !table))))
        return LORA_EINVAL;
    size_t most = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (!P->has(seqs[i])) return LORA_EINVAL;
        most = std::max(most, P->seqs[(size_t)seqs[i]].pages.size());
    }
    *n_columns = (int32_t)most;
    if ((int64_t)most > ld_table) return LORA_ECAPACITY;
    for (int32_t i = 0; i < n; ++i) {
        const lora_kv_pages::Seq& s = P->seqs[(size_t)seqs[i]];
        kv_len[i] = s.tokens;
        if (ld_table == 0) continue;
        int32_t* row = table + i * ld_table;
        std::fill(std::copy(s.pages.begin(), s.pages.end(), row), row + ld_table, 0);
    }
    return LORA_OK;
}

extern "C" int32_t lora_kv_pages_stats(const lora_kv_pages_t* P, int32_t* n_free, int32_t* n_shared, int32_t* end) {
    if (!P) return LORA_EINVAL;
    int32_t shared = 0, last = 0;
    for (int32_t p = 0; p < P->n_pages; ++p) {
        shared += P->users[(size_t)p] > 1;
        if (P->users[(size_t)p] > 0) last = p + 1;
    }
    if (n_free) *n_free = (int32_t)P->free_pages.size();
    if (n_shared) *n_shared = shared;
    if (end) *end = last;
    return LORA_OK;
}
