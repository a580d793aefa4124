// Host-side pool of a paged cache's pages (HPD-Parsing, part 2: shared-prefix KV reuse -- content branches fork from what
// their parent has read, and shared KV is freed by reference count -- for caches that live in pages).
//
// A page holds the rows of one or more sequences; a fork shares all of its parent's.  Only a sequence's last page is ever
// written to, by append: when others hold it too, the sequence gets a copy first (copy on write), which the caller makes.
#include <stdarg.h>
#include <stdio.h>

#include <exception>
#include <mutex>
#include <vector>

#include "fx_internal.h"

namespace {

int pool_error(fx_status st, const char* fmt, ...)
{
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    fx::set_error(st, buf);
    return -1;
}

struct Sequence {
    bool live = false;
    int len = 0;
    std::vector<int32_t> pages;
};

}  // namespace

struct fx_page_pool {
    std::mutex mu;
    int page_rows = 0, max_pages = 0;
    std::vector<int> refs;        // of every page
    std::vector<int32_t> free;    // the next page to give out is the last
    std::vector<Sequence> seqs;

    Sequence* find(int seq)
    {
        if (seq < 0 || seq >= (int)seqs.size() || !seqs[seq].live) {
            pool_error(FX_ERR_INVALID_ARG, "sequence %d is not live", seq);
            return nullptr;
        }
        return &seqs[seq];
    }
    int open()
    {
        for (int i = 0; i < (int)seqs.size(); ++i)
            if (!seqs[i].live) return i;
        return pool_error(FX_ERR_UNSUPPORTED, "all %d sequences are taken", (int)seqs.size());
    }
    int drop(Sequence& s, size_t keep)   // pages from number `keep` on; how many became free
    {
        int n = 0;
        while (s.pages.size() > keep) {
            const int32_t pg = s.pages.back();
            s.pages.pop_back();
            if (--refs[pg] == 0) {
                free.push_back(pg);   // (room for all pages was reserved)
                ++n;
            }
        }
        return n;
    }
};

extern "C" {

fx_page_pool* fx_page_pool_create(int n_pages, int page_rows, int max_seqs, int max_pages)
{
    if (n_pages < 1 || page_rows < 1 || max_seqs < 1 || max_pages < 1 || (int64_t)max_pages * page_rows > 2147483647) {
        pool_error(FX_ERR_INVALID_ARG, "need n_pages, page_rows, max_seqs, max_pages >= 1 and rows of a sequence below 2^31");
        return nullptr;
    }
    fx_page_pool* p = nullptr;
    try {
        p = new fx_page_pool;
        p->page_rows = page_rows;
        p->max_pages = max_pages;
        p->refs.assign(n_pages, 0);
        p->free.reserve(n_pages);
        for (int i = n_pages - 1; i >= 0; --i) p->free.push_back(i);
        p->seqs.resize(max_seqs);
    } catch (const std::exception&) {
        delete p;
        pool_error(FX_ERR_INVALID_ARG, "no memory for a pool of %d pages and %d sequences", n_pages, max_seqs);
        return nullptr;
    }
    return p;
}

void fx_page_pool_destroy(fx_page_pool* pool) { delete pool; }

int fx_page_pool_open(fx_page_pool* pool)
{
    if (!pool) return pool_error(FX_ERR_INVALID_ARG, "pool is NULL");
    std::lock_guard<std::mutex> lock(pool->mu);
    const int id = pool->open();
    if (id >= 0) {
        pool->seqs[id].live = true;
        pool->seqs[id].len = 0;
    }
    return id;
}

int fx_page_pool_append(fx_page_pool* pool, int seq, int n, int32_t* copy_src, int32_t* copy_dst)
{
    if (!pool || n < 0 || !copy_src || !copy_dst)
        return pool_error(FX_ERR_INVALID_ARG, "pool, copy_src or copy_dst is NULL or n < 0");
    std::lock_guard<std::mutex> lock(pool->mu);
    Sequence* s = pool->find(seq);
    if (!s) return -1;
    const int64_t len = (int64_t)s->len + n, need = (len + pool->page_rows - 1) / pool->page_rows;
    if (need > pool->max_pages)
        return pool_error(FX_ERR_UNSUPPORTED, "sequence %d: %lld rows, %d pages at most", seq, (long long)len, pool->max_pages);
    // the page that the first new row goes to, when the sequence has it already
    const bool copy = n > 0 && s->len % pool->page_rows != 0 && pool->refs[s->pages.back()] > 1;
    const int64_t fresh = need - (int64_t)s->pages.size() + (copy ? 1 : 0);
    if (fresh > (int64_t)pool->free.size())
        return pool_error(FX_ERR_UNSUPPORTED, "sequence %d: %lld pages wanted, %lld free", seq, (long long)fresh,
                          (long long)pool->free.size());
    try {
        s->pages.reserve(need);
    } catch (const std::exception&) {
        return pool_error(FX_ERR_UNSUPPORTED, "no memory for a table of %lld pages", (long long)need);
    }
    auto take = [&] {
        const int32_t pg = pool->free.back();
        pool->free.pop_back();
        pool->refs[pg] = 1;
        return pg;
    };
    *copy_src = *copy_dst = -1;
    if (copy) {
        *copy_src = s->pages.back();
        --pool->refs[s->pages.back()];
        *copy_dst = s->pages.back() = take();
    }
    while ((int64_t)s->pages.size() < need) s->pages.push_back(take());
    s->len = (int)len;
    return copy ? 1 : 0;
}

int fx_page_pool_fork(fx_page_pool* pool, int seq)
{
    if (!pool) return pool_error(FX_ERR_INVALID_ARG, "pool is NULL");
    std::lock_guard<std::mutex> lock(pool->mu);
    Sequence* s = pool->find(seq);
    if (!s) return -1;
    const int id = pool->open();
    if (id < 0) return -1;
    Sequence& t = pool->seqs[id];
    try {
        t.pages = s->pages;
    } catch (const std::exception&) {
        t.pages.clear();
        return pool_error(FX_ERR_UNSUPPORTED, "no memory for a table of %lld pages", (long long)s->pages.size());
    }
    t.live = true;
    t.len = s->len;
    for (const int32_t pg : t.pages) ++pool->refs[pg];
    return id;
}

int fx_page_pool_truncate(fx_page_pool* pool, int seq, int n)
{
    if (!pool) return pool_error(FX_ERR_INVALID_ARG, "pool is NULL");
    std::lock_guard<std::mutex> lock(pool->mu);
    Sequence* s = pool->find(seq);
    if (!s) return -1;
    if (n < 0 || n > s->len) return pool_error(FX_ERR_INVALID_ARG, "sequence %d has %d rows, not %d", seq, s->len, n);
    s->len = n;
    return pool->drop(*s, ((size_t)n + pool->page_rows - 1) / pool->page_rows);
}

int fx_page_pool_release(fx_page_pool* pool, int seq)
{
    if (!pool) return pool_error(FX_ERR_INVALID_ARG, "pool is NULL");
    std::lock_guard<std::mutex> lock(pool->mu);
    Sequence* s = pool->find(seq);
    if (!s) return -1;
    s->live = false;
    s->len = 0;
    return pool->drop(*s, 0);
}

int fx_page_pool_length(fx_page_pool* pool, int seq)
{
    if (!pool) return pool_error(FX_ERR_INVALID_ARG, "pool is NULL");
    std::lock_guard<std::mutex> lock(pool->mu);
    Sequence* s = pool->find(seq);
    return s ? s->len : -1;
}

int fx_page_pool_free_pages(fx_page_pool* pool)
{
    if (!pool) return pool_error(FX_ERR_INVALID_ARG, "pool is NULL");
    std::lock_guard<std::mutex> lock(pool->mu);
    return (int)pool->free.size();
}

int fx_page_pool_batch(fx_page_pool* pool, const int32_t* seqs, int n, int32_t* table, int32_t* len)
{
    if (!pool || n < 0 || (n > 0 && (!seqs || !table || !len)))
        return pool_error(FX_ERR_INVALID_ARG, "pool or an array is NULL, or n < 0");
    std::lock_guard<std::mutex> lock(pool->mu);
    for (int i = 0; i < n; ++i)
        if (!pool->find(seqs[i])) return -1;
    for (int i = 0; i < n; ++i) {
        const Sequence& s = pool->seqs[seqs[i]];
        int32_t* row = table + (int64_t)i * pool->max_pages;
        for (int j = 0; j < pool->max_pages; ++j) row[j] = j < (int)s.pages.size() ? s.pages[j] : -1;
        len[i] = s.len;
    }
    return n;
}

}  // extern "C"
