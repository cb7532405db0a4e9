// Which sequence owns which page of a paged cache: reference counts, copy on
// write, and the page copies the device has to make.  Host only.
//
// A batch of copies handed out together runs in one launch, in no order, so
// no page of it may be both read and written.  Two rules see to that: the
// page a queued copy reads is held by the queue (it cannot become free and be
// given away), and a copy from a page that is itself still to be written
// reads that page's source instead.
//
// Copies run before the appends of their step.  So one that reads rows which
// were reserved in the same step would miss them: a sequence is forked after
// its reserve, and one of the two grows.  The manager does not see the appends;
// rows count as written once a later call handed out the copies or the tables
// they are appended by, and until then such a copy is not handed out.
#include <algorithm>
#include <cstdint>
#include <exception>
#include <vector>

#include "bsa.h"
#include "bsa_errors.h"

struct bsa_pages_s {
    struct Seq {
        std::vector<int32_t> pages;
        int64_t length = 0;
    };
    struct Copy {
        int32_t from, to;
        uint64_t step;               // reads rows reserved in it; 0: none
    };
    struct Fresh {
        uint64_t step = 0;
        int32_t row = 0;
    };
    int32_t page = 0, width = 0;
    uint64_t step = 1;               // ends when copies or tables are handed out
    std::vector<int32_t> refs;       // holders of each page
    std::vector<Fresh> fresh;        // of each page: lowest row reserved in a step
    std::vector<int32_t> free_list;  // taken from the back
    std::vector<Seq> seqs;
    std::vector<Copy> copies;

    // Both vectors never grow past their reserved sizes, so neither throws.
    void release(int32_t p) {
        if (--refs[p] > 0) return;
        free_list.push_back(p);
    }
    int32_t fresh_row(int32_t p) const {            // rows from it on are not written yet
        return fresh[size_t(p)].step == step ? fresh[size_t(p)].row : page;
    }
    void drop(int32_t p) {           // a sequence lets go of its page
        if (refs[p] == 1)
            for (size_t i = 0; i < copies.size(); ++i)
                if (copies[i].to == p) {        // nobody will read it
                    const int32_t from = copies[i].from;
                    copies.erase(copies.begin() + int64_t(i));
                    release(from);
                    break;
                }
        release(p);
    }
};

namespace {

using bsa::fail;
using bsa::ok;

bsa_status check_seq(bsa_pages p, int32_t seq) {
    if (p == nullptr) return fail(BSA_ERR_INVALID_ARG, "pages is NULL");
    if (seq < 0 || size_t(seq) >= p->seqs.size())
        return fail(BSA_ERR_INVALID_ARG, "sequence %d is outside [0, %zu)", seq, p->seqs.size());
    return BSA_OK;
}

}  // namespace

extern "C" {

bsa_status bsa_pages_create(int64_t num_pages, int32_t page, int32_t max_seqs,
                            int32_t table_width, bsa_pages *pages) {
    if (pages == nullptr) return fail(BSA_ERR_INVALID_ARG, "pages is NULL");
    *pages = nullptr;
    if (num_pages < 1 || num_pages > 0x7fffffff || max_seqs < 1 || table_width < 1)
        return fail(BSA_ERR_INVALID_ARG, "num_pages, max_seqs and table_width must be >= 1 (and fit int32)");
    if (page != 16 && page != 32 && page != 64 && page != 128)
        return fail(BSA_ERR_UNSUPPORTED, "page must be 16, 32, 64 or 128 (got %d)", page);
    try {
        bsa_pages p = new bsa_pages_s;
        try {
            p->page = page;
            p->width = table_width;
            p->refs.assign(size_t(num_pages), 0);
            p->fresh.resize(size_t(num_pages));
            p->free_list.reserve(size_t(num_pages));
            for (int64_t i = num_pages; i-- > 0;) p->free_list.push_back(int32_t(i));
            p->seqs.resize(size_t(max_seqs));
        } catch (...) {
            delete p;
            throw;
        }
        *pages = p;
    } catch (const std::exception &) {
        return fail(BSA_ERR_CUDA, "out of host memory");
    }
    return ok();
}

bsa_status bsa_pages_destroy(bsa_pages pages) {
    delete pages;
    return ok();
}

bsa_status bsa_pages_reserve(bsa_pages pages, int32_t seq, int64_t tokens) {
    if (bsa_status st = check_seq(pages, seq); st != BSA_OK) return st;
    auto &s = pages->seqs[size_t(seq)];
    if (tokens < 0 || tokens > 0x7fffffff - s.length)
        return fail(BSA_ERR_INVALID_ARG, "tokens must be >= 0 and the length at most 2^31 - 1");
    if (tokens == 0) return ok();
    const int64_t page = pages->page;
    const size_t want = size_t((s.length + tokens + page - 1) / page);
    if (want > size_t(pages->width))
        return fail(BSA_ERR_WORKSPACE, "sequence %d needs %zu pages, its table holds %d", seq, want,
                    pages->width);
    // shared with another sequence (a queued copy reads it before the append)
    int32_t holders = s.length % page != 0 ? pages->refs[size_t(s.pages.back())] : 1;
    if (holders > 1)
        for (const auto &c : pages->copies) holders -= c.from == s.pages.back();
    const bool split = holders > 1;
    const size_t fresh = want - s.pages.size() + (split ? 1 : 0);
    if (fresh > pages->free_list.size())
        return fail(BSA_ERR_WORKSPACE, "%zu pages wanted, %zu are free", fresh, pages->free_list.size());
    try {
        s.pages.reserve(want);
        if (split) pages->copies.reserve(pages->copies.size() + 1);
    } catch (const std::exception &) {
        return fail(BSA_ERR_CUDA, "out of host memory");
    }
    const auto take = [&] {
        const int32_t p = pages->free_list.back();
        pages->free_list.pop_back();
        pages->refs[size_t(p)] = 1;
        pages->fresh[size_t(p)] = {pages->step, 0};
        return p;
    };
    const int32_t rows = int32_t(s.length % page);      // of the last page, if partly filled
    int32_t unwritten = rows;
    if (rows != 0) unwritten = std::min(rows, pages->fresh_row(s.pages.back()));
    if (split) {
        const int32_t old = s.pages.back(), p = take();
        int32_t from = old;
        for (const auto &c : pages->copies)
            if (c.to == old) from = c.from;     // still to be written itself
        pages->copies.push_back({from, p, unwritten < rows ? pages->step : 0});
        ++pages->refs[size_t(from)];            // held until the copy is taken
        s.pages.back() = p;
        pages->drop(old);
    }
    if (rows != 0) pages->fresh[size_t(s.pages.back())] = {pages->step, unwritten};
    while (s.pages.size() < want) s.pages.push_back(take());
    s.length += tokens;
    return ok();
}

bsa_status bsa_pages_fork(bsa_pages pages, int32_t from, int32_t to) {
    if (bsa_status st = check_seq(pages, from); st != BSA_OK) return st;
    if (bsa_status st = check_seq(pages, to); st != BSA_OK) return st;
    auto &a = pages->seqs[size_t(from)], &b = pages->seqs[size_t(to)];
    if (from == to || b.length != 0)
        return fail(BSA_ERR_INVALID_ARG, "sequence %d is not an empty other one", to);
    try {
        b.pages = a.pages;
    } catch (const std::exception &) {
        return fail(BSA_ERR_CUDA, "out of host memory");
    }
    b.length = a.length;
    for (int32_t p : b.pages) ++pages->refs[size_t(p)];
    return ok();
}

bsa_status bsa_pages_truncate(bsa_pages pages, int32_t seq, int64_t length) {
    if (bsa_status st = check_seq(pages, seq); st != BSA_OK) return st;
    auto &s = pages->seqs[size_t(seq)];
    if (length < 0 || length > s.length)
        return fail(BSA_ERR_INVALID_ARG, "length must be in [0, %lld]", (long long)s.length);
    const size_t keep = size_t((length + pages->page - 1) / pages->page);
    while (s.pages.size() > keep) {
        const int32_t p = s.pages.back();
        s.pages.pop_back();
        pages->drop(p);
    }
    s.length = length;
    return ok();
}

bsa_status bsa_pages_take_copies(bsa_pages pages, int32_t *pairs, int64_t capacity,
                                 int64_t *count) {
    if (pages == nullptr || count == nullptr)
        return fail(BSA_ERR_INVALID_ARG, "pages or count is NULL");
    *count = int64_t(pages->copies.size());
    if (pairs == nullptr) return ok();
    if (capacity < *count)
        return fail(BSA_ERR_WORKSPACE, "%lld copies are queued", (long long)*count);
    for (const auto &c : pages->copies)
        if (c.step == pages->step)
            return fail(BSA_ERR_INVALID_ARG,
                        "the copy of page %d to %d would miss tokens reserved since the last "
                        "take_copies or tables: append them first and call tables, or free the fork",
                        c.from, c.to);
    ++pages->step;
    for (const auto &c : pages->copies) {
        *pairs++ = c.from;
        *pairs++ = c.to;
    }
    for (const auto &c : pages->copies) pages->release(c.from);
    pages->copies.clear();
    return ok();
}

bsa_status bsa_pages_compact(bsa_pages pages, int32_t *pairs, int64_t capacity, int64_t *count) {
    if (pages == nullptr || count == nullptr)
        return fail(BSA_ERR_INVALID_ARG, "pages or count is NULL");
    if (!pages->copies.empty())
        return fail(BSA_ERR_INVALID_ARG, "copies are queued: take them first");
    auto &refs = pages->refs;
    const int64_t total = int64_t(refs.size());
    const int64_t used = total - int64_t(pages->free_list.size());
    int64_t moves = 0;
    for (int64_t p = used; p < total; ++p) moves += refs[size_t(p)] > 0;
    *count = moves;
    if (pairs == nullptr) return ok();
    if (capacity < moves) return fail(BSA_ERR_WORKSPACE, "%lld pages have to move", (long long)moves);
    std::vector<int32_t> at;
    try {
        at.resize(size_t(total - used));        // new place of page used + i
    } catch (const std::exception &) {
        return fail(BSA_ERR_CUDA, "out of host memory");
    }
    int64_t hole = 0;
    for (int64_t p = used; p < total; ++p) {
        if (refs[size_t(p)] == 0) continue;
        while (refs[size_t(hole)] != 0) ++hole;
        *pairs++ = int32_t(p);
        *pairs++ = int32_t(hole);
        refs[size_t(hole)] = refs[size_t(p)];
        refs[size_t(p)] = 0;
        pages->fresh[size_t(hole)] = pages->fresh[size_t(p)];
        at[size_t(p - used)] = int32_t(hole);
    }
    for (auto &s : pages->seqs)
        for (int32_t &p : s.pages)
            if (p >= used) p = at[size_t(p - used)];
    pages->free_list.clear();
    for (int64_t p = total; p-- > used;) pages->free_list.push_back(int32_t(p));
    return ok();
}

bsa_status bsa_pages_tables(bsa_pages pages, int32_t *table, int32_t *lengths) {
    if (pages == nullptr) return fail(BSA_ERR_INVALID_ARG, "pages is NULL");
    if (table != nullptr || lengths != nullptr) ++pages->step;
    for (size_t s = 0; s < pages->seqs.size(); ++s) {
        const auto &q = pages->seqs[s];
        if (table != nullptr) {
            int32_t *row = table + int64_t(s) * pages->width;
            for (size_t i = 0; i < size_t(pages->width); ++i)
                row[i] = i < q.pages.size() ? q.pages[i] : -1;
        }
        if (lengths != nullptr) lengths[s] = int32_t(q.length);
    }
    return ok();
}

int64_t bsa_pages_free_pages(bsa_pages pages) {
    if (pages == nullptr) return -int64_t(fail(BSA_ERR_INVALID_ARG, "pages is NULL"));
    return int64_t(pages->free_list.size());
}

}  // extern "C"
