// Host-side accounting of the pages of a paged memory (txl_page_pool in
// include/txl.h): a stack of free pages and the number of users of each page.
// Plain arithmetic on the caller's arrays; nothing here touches the device.
#include "txl.h"

namespace {

bool pool_ok(const txl_page_pool *p)
{
    return p && p->free_list && p->users && p->n_pages >= 0 && p->n_free >= 0 &&
           p->n_free <= p->n_pages;
}

// Every id in range and in use.
bool in_use(const txl_page_pool *p, const int *pages, int n)
{
    if (n < 0 || (n > 0 && !pages)) return false;
    for (int i = 0; i < n; ++i)
        if (pages[i] < 0 || pages[i] >= p->n_pages || p->users[pages[i]] < 1) return false;
    return true;
}

} // namespace

extern "C" int txl_page_pool_init(txl_page_pool *p, int n_pages, int *free_list, int *users)
{
    if (!p || n_pages < 0 || !free_list || !users) return TXL_ERR_INVALID_ARG;
    p->n_pages = p->n_free = n_pages;
    p->free_list = free_list;
    p->users = users;
    for (int i = 0; i < n_pages; ++i) {
        free_list[i] = n_pages - 1 - i;  // page 0 is handed out first
        users[i] = 0;
    }
    return TXL_OK;
}

extern "C" int txl_page_pool_alloc(txl_page_pool *p, int *pages, int n)
{
    if (!pool_ok(p) || n < 0 || (n > 0 && !pages)) return TXL_ERR_INVALID_ARG;
    if (n > p->n_free) return TXL_ERR_SHAPE;
    for (int i = 0; i < n; ++i) {
        pages[i] = p->free_list[--p->n_free];
        p->users[pages[i]] = 1;
    }
    return TXL_OK;
}

extern "C" int txl_page_pool_retain(txl_page_pool *p, const int *pages, int n)
{
    if (!pool_ok(p) || !in_use(p, pages, n)) return TXL_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) ++p->users[pages[i]];
    return TXL_OK;
}

extern "C" int txl_page_pool_release(txl_page_pool *p, const int *pages, int n, int *n_freed)
{
    if (!pool_ok(p) || !in_use(p, pages, n)) return TXL_ERR_INVALID_ARG;
    // A page named more often than it has users: take the counts back, change
    // nothing.
    int done = 0;
    while (done < n && p->users[pages[done]] > 0) --p->users[pages[done++]];
    if (done < n) {
        while (done > 0) ++p->users[pages[--done]];
        return TXL_ERR_INVALID_ARG;
    }
    int freed = 0;
    for (int i = n - 1; i >= 0; --i) {
        // a page named twice is put on the list once: marked by -1 until the end
        if (p->users[pages[i]] != 0) continue;
        p->users[pages[i]] = -1;
        p->free_list[p->n_free++] = pages[i];
        ++freed;
    }
    for (int i = 0; i < freed; ++i) p->users[p->free_list[p->n_free - 1 - i]] = 0;
    if (n_freed) *n_freed = freed;
    return TXL_OK;
}
