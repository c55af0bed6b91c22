/*
 * prefix_scan_pages.h -- C ABI for the pages of a cache: pools of equal pages
 * (keys and values of some tokens, or the recurrent state of a sequence,
 * prefix_scan_delta.h), shared by reference counts and named by page tables.
 * Handing out the lowest free pages and moving pages together are scans and
 * stream compactions (prefix_scan.h) over the counts; here they come fused
 * with what they are for.
 *
 *   pools     npools device arrays (one per layer, say) of `pages` pages each,
 *             page i of a pool at data + i * page_bytes
 *   refcount  device int32 [pages]: how many table entries hold each page; a
 *             page whose count is 0 or less is free
 *   table     device int32 [rows, width], contiguous: row r's pages in order,
 *             -1 where there is none.  Indices outside [0, pages) are treated
 *             as -1.
 *   lengths   device int32 [rows]: tokens of each row, clamped to
 *             [0, width * page_tokens]
 *
 * Results do not depend on scheduling: pages are handed out lowest first, in
 * the order of rows and of places in a row.  Counts change by integer atomics.
 *
 * Conventions as in prefix_scan.h: device pointers owned by the caller, work
 * enqueued on `stream` without waiting, nothing allocated or kept, calls can be
 * captured in CUDA graphs; errors found on the host are returned before
 * anything is enqueued (PS_ERR_INVALID_ARG, PS_ERR_WORKSPACE_TOO_SMALL,
 * PS_ERR_OVERLAP, PS_ERR_CUDA).  A workspace of
 * ps_pages_workspace_size(rows, pages) bytes, 256-byte aligned, serves every
 * call and needs no preparation; calls that may run at the same time must not
 * share one.  rows, width and pages are at most 2^31 - 1 together with
 * rows * width; pages of one call are copied whole, in any order.
 */
#ifndef PREFIX_SCAN_PAGES_H
#define PREFIX_SCAN_PAGES_H

#include "prefix_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PS_PAGES_MAX_POOLS 128

typedef struct ps_page_pool {
    void *data;
    int64_t page_bytes;
} ps_page_pool;

/* Bytes of workspace for tables of up to `rows` rows and pools of `pages` pages. */
size_t ps_pages_workspace_size(int64_t rows, int64_t pages);

/*
 * Copies page src[i] to page dst[i] of every pool, i < n (device arrays).
 * Pairs with an index outside [0, pages) are left out.  No page may be
 * written twice, or written and read.
 */
ps_status ps_pages_copy(const ps_page_pool *pools, int npools, int64_t pages, const int32_t *src,
                        const int32_t *dst, int64_t n, ps_stream_t stream);

/*
 * Forks: row i of the new table becomes a branch of row parents[i] of `table`
 * (any row any number of times; an index outside [0, rows) gives an empty
 * row).  Whole pages are shared, their counts raised; a part-filled last page,
 * which parent and branch will both write to, is copied to a free page.
 *   new_table    [new_rows, width], new_lengths [new_rows]
 *   missing      device int32 [1]: how many last pages found no free page (those
 *                places are -1); may be NULL
 */
ps_status ps_pages_fork(const int32_t *table, const int32_t *lengths, int64_t rows, int64_t width,
                        const int32_t *parents, int64_t new_rows, int32_t page_tokens, int32_t *refcount,
                        const ps_page_pool *pools, int npools, int64_t pages, int32_t *new_table,
                        int32_t *new_lengths, int32_t *missing, void *ws, size_t ws_bytes, ps_stream_t stream);

/*
 * Grows: gives row r the pages it needs to hold new_lengths[r] tokens instead
 * of lengths[r], at the places of its row that these add and that hold none.
 *   missing  device int32 [1]: places that found no free page, or that lie past
 *            the table's width; may be NULL
 */
ps_status ps_pages_grow(int32_t *table, const int32_t *lengths, const int32_t *new_lengths, int64_t rows,
                        int64_t width, int32_t page_tokens, int32_t *refcount, int64_t pages, int32_t *missing,
                        void *ws, size_t ws_bytes, ps_stream_t stream);

/*
 * Frees: lets go of every page of the rows with flags[r] != 0 (all rows if
 * flags is NULL): their counts fall, their places become -1.
 */
ps_status ps_pages_free(int32_t *table, int64_t rows, int64_t width, const uint8_t *flags, int32_t *refcount,
                        int64_t pages, ps_stream_t stream);

/*
 * Compacts: moves pages so that the m pages in use are pages 0 .. m-1.  Pages
 * below m stay; the i-th page in use at or above m moves to the i-th free page
 * below m, in all pools; counts and the table's entries follow.  Entries that
 * name a free page become -1.
 *   used  device int32 [1] receiving m; may be NULL
 */
ps_status ps_pages_compact(int32_t *table, int64_t rows, int64_t width, int32_t *refcount,
                           const ps_page_pool *pools, int npools, int64_t pages, int32_t *used, void *ws,
                           size_t ws_bytes, ps_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PREFIX_SCAN_PAGES_H */
