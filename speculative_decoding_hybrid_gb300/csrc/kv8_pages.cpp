// Page tables of the paged key/value cache: host integers over a gdn_pool
// whose slots are the cache's pages ("Run chained MTP drafting in the batch
// Engine", RC4 evidence: paged Engine; "Native three-step MTP", Results:
// shared-prefix protection, duplicate-slot release).  Every call checks first
// and changes the pool and the tables afterwards, so an error leaves both as
// they were.
#include <stdint.h>

#include <new>
#include <vector>

#include "gdnspec.h"

namespace {

bool page_tokens_ok(int32_t t) { return t == 16 || t == 32 || t == 64 || t == 128; }
bool held(const gdn_pool *p, int32_t s) { return s >= 0 && s < p->num_slots && p->refcount[s] > 0; }

}  // namespace

extern "C" int kv8_pages_reserve(gdn_pool *pool, int32_t *table, int32_t table_cap, int32_t *n_pages, int32_t len,
                                 int32_t n_new, int32_t page_tokens, int32_t *copy_src, int32_t *copy_dst,
                                 int32_t *n_copy) {
    if (!pool || !n_pages || !copy_src || !copy_dst || !n_copy || (table_cap > 0 && !table)) return GDN_ERR_NULL;
    if (!page_tokens_ok(page_tokens) || table_cap < 0 || len < 0 || n_new < 0 || *n_pages < 0 || *n_pages > table_cap)
        return GDN_ERR_ARG;
    const int64_t have = *n_pages, T = page_tokens;
    const int64_t need = (int64_t(len) + n_new + T - 1) / T;
    if ((int64_t(len) + T - 1) / T > have || need > table_cap) return GDN_ERR_ARG;
    for (int64_t i = 0; i < have; ++i)
        if (!held(pool, table[i])) return GDN_ERR_ARG;
    // Pages that the new positions would write into and somebody else holds
    // too.  An unfinished page is copied; a page kept past the end of the
    // positions (after a rollback) has nothing to keep and is replaced.
    const int64_t first = len / T, last = need < have ? need : have;
    int64_t fresh = need > have ? need - have : 0;
    if (n_new > 0)
        for (int64_t i = first; i < last; ++i) fresh += pool->refcount[table[i]] > 1;
    if (fresh > pool->free_count) return GDN_ERR_NO_SLOT;
    *n_copy = 0;
    if (n_new > 0)
        for (int64_t i = first; i < last; ++i)
            if (pool->refcount[table[i]] > 1) {
                int32_t s = -1;
                gdn_pool_alloc(pool, &s);
                if (i * T < len) {
                    *copy_src = table[i];
                    *copy_dst = s;
                    *n_copy = 1;
                }
                gdn_pool_release(pool, table[i]);
                table[i] = s;
            }
    for (int64_t i = have; i < need; ++i) gdn_pool_alloc(pool, &table[i]);
    if (need > have) *n_pages = int32_t(need);
    return GDN_OK;
}

extern "C" int kv8_pages_fork(gdn_pool *pool, const int32_t *src_table, int32_t src_pages, int32_t len,
                              int32_t page_tokens, int32_t *dst_table, int32_t table_cap, int32_t *dst_pages,
                              int32_t *copy_src, int32_t *copy_dst, int32_t *n_copy) {
    if (!pool || !dst_pages || !copy_src || !copy_dst || !n_copy || (src_pages > 0 && !src_table) ||
        (table_cap > 0 && !dst_table))
        return GDN_ERR_NULL;
    if (!page_tokens_ok(page_tokens) || src_pages < 0 || len < 0 || table_cap < 0 || *dst_pages != 0)
        return GDN_ERR_ARG;
    const int64_t T = page_tokens, whole = len / T, need = (int64_t(len) + T - 1) / T;
    if (need > src_pages || need > table_cap) return GDN_ERR_ARG;
    for (int64_t i = 0; i < need; ++i)
        if (!held(pool, src_table[i])) return GDN_ERR_ARG;
    if (need > whole && pool->free_count == 0) return GDN_ERR_NO_SLOT;
    *n_copy = 0;
    for (int64_t i = 0; i < whole; ++i) {
        gdn_pool_share(pool, src_table[i]);
        dst_table[i] = src_table[i];
    }
    if (need > whole) {
        gdn_pool_alloc(pool, &dst_table[whole]);
        *copy_src = src_table[whole];
        *copy_dst = dst_table[whole];
        *n_copy = 1;
    }
    *dst_pages = int32_t(need);
    return GDN_OK;
}

extern "C" int kv8_pages_free(gdn_pool *pool, int32_t *table, int32_t *n_pages) {
    if (!pool || !n_pages || (*n_pages > 0 && !table)) return GDN_ERR_NULL;
    if (*n_pages < 0) return GDN_ERR_ARG;
    // a page named twice needs two references (checked by taking them off)
    int32_t i = 0;
    for (; i < *n_pages; ++i) {
        if (!held(pool, table[i])) break;
        pool->refcount[table[i]]--;
    }
    const bool all = i == *n_pages;
    for (int32_t j = 0; j < i; ++j) pool->refcount[table[j]]++;
    if (!all) return GDN_ERR_ARG;
    for (int32_t j = 0; j < *n_pages; ++j) {
        gdn_pool_release(pool, table[j]);
        table[j] = -1;
    }
    *n_pages = 0;
    return GDN_OK;
}

extern "C" int kv8_pages_compact(gdn_pool *pool, int32_t n_tables, int32_t *tables, int32_t table_stride,
                                 const int32_t *n_pages, int32_t *move_src, int32_t *move_dst, int32_t *n_moves) {
    if (!pool || !n_moves || !move_src || !move_dst || (n_tables > 0 && (!tables || !n_pages))) return GDN_ERR_NULL;
    if (n_tables < 0 || table_stride < 0) return GDN_ERR_ARG;
    const int32_t n = pool->num_slots;
    std::vector<int32_t> seen, to;
    try {
        seen.assign(size_t(n), 0);
        to.assign(size_t(n), -1);
    } catch (const std::bad_alloc &) {
        return GDN_ERR_WORKSPACE;
    }
    for (int32_t r = 0; r < n_tables; ++r) {
        if (n_pages[r] < 0 || n_pages[r] > table_stride) return GDN_ERR_ARG;
        for (int32_t i = 0; i < n_pages[r]; ++i) {
            const int32_t s = tables[int64_t(r) * table_stride + i];
            if (!held(pool, s)) return GDN_ERR_ARG;
            seen[size_t(s)]++;
        }
    }
    int32_t live = 0;
    for (int32_t s = 0; s < n; ++s) {
        if (seen[size_t(s)] != pool->refcount[s]) return GDN_ERR_ARG;
        live += pool->refcount[s] > 0;
    }
    int32_t hole = 0, moves = 0;
    for (int32_t s = live; s < n; ++s) {
        if (pool->refcount[s] == 0) continue;
        while (pool->refcount[hole] > 0) ++hole;  // one below `live` for every live page past it
        move_src[moves] = s;
        move_dst[moves++] = hole;
        to[size_t(s)] = hole;
        pool->refcount[hole] = pool->refcount[s];
        pool->refcount[s] = 0;
    }
    for (int32_t r = 0; r < n_tables; ++r)
        for (int32_t i = 0; i < n_pages[r]; ++i) {
            int32_t &e = tables[int64_t(r) * table_stride + i];
            if (to[size_t(e)] >= 0) e = to[size_t(e)];
        }
    pool->free_head = 0;
    pool->free_count = n - live;
    for (int32_t i = 0; i < n - live; ++i) pool->free_fifo[i] = live + i;
    *n_moves = moves;
    return GDN_OK;
}
