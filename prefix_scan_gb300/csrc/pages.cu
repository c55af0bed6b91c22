// pages.cu -- pages of a cache: copy, fork, reorder, grow, free, compact
// (include/prefix_scan_pages.h).
//
// Each call that hands out or moves pages is a plan and a move.  The plan is
// one CTA of 1024 threads that scans the reference counts in tiles of 16384
// pages (ranks of free or used pages from ballots and a sum over the warps) and
// writes lists into the workspace; a plan that hands out pages ends at the first
// tile that holds enough of them.  The move is a grid of CTAs
// that copy pieces of pages and rewrite the tables.  Moves are bound by memory:
// a moved page is read once and written once.  Compacting 16384 pages of two pools
// of 32 KiB, of which 3585 move: 100 us, the move 75 of it at 6.3 TB/s.  Smaller calls
// are bound by their launches and the host: 37 pages copied in 10 us.
#include <climits>
#include <cstdint>

#include "prefix_scan_pages.h"
#include "scan_internal.h"

namespace ps {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanItems = 16;                             // pages of a thread in a tile
constexpr int kPlanTile = kPlanThreads * kPlanItems;
constexpr int kMoveThreads = 256;
constexpr int kPiece = 16384;                              // bytes of a page that a CTA moves at a time
constexpr int kMoveCtas = 152 * 4;

struct Pools {
    ps_page_pool pool[PS_PAGES_MAX_POOLS];
    int n;
    int pieces;                                            // pieces of a page over all pools
};

// Workspace: [0] how many entries the lists hold; then ranks [rows], and lists of up to `pages`.
struct PlanSpace {
    int32_t *head, *rank, *list, *from, *to;
};
__host__ __device__ inline size_t ints(size_t n) { return (n + 63) / 64 * 64; }
__host__ __device__ inline PlanSpace plan_space(void *ws, long long rows, long long pages) {
    int32_t *p = static_cast<int32_t *>(ws);
    PlanSpace s;
    s.head = p;
    s.rank = p + 64;
    s.list = s.rank + ints((size_t)rows);
    s.from = s.list + ints((size_t)pages);
    s.to = s.from + ints((size_t)pages);
    return s;
}

// Exclusive sum over the block's threads; `total` receives the sum.
__device__ __forceinline__ int block_exclusive(int x, int *warps, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    __syncthreads();   // the last call's sums have been read
    if (lane == 31) warps[warp] = s;
    __syncthreads();
    const int w = warps[lane];
    int t = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, t, d);
        if (lane >= d) t += y;
    }
    total = __shfl_sync(0xffffffffu, t, 31);
    return s - x + __shfl_sync(0xffffffffu, t - w, warp);
}

// A tile's pages by warps: warp w holds pages 512 w ... 512 w + 511 of it, lane l of its item i page 32 i + l, so loads
// and the lists' stores are whole lines, and a page's rank comes from the ballots of its warp.
__device__ __forceinline__ long long tile_page(long long base, int item) {
    return base + (threadIdx.x >> 5) * (32 * kPlanItems) + item * 32 + (threadIdx.x & 31);
}
// Bit l of mask[i]: whether page 32 i + l of the warp's holds `is_used`; pages past the end hold neither.
__device__ __forceinline__ void load_masks(uint32_t (&mask)[kPlanItems], const int32_t *refcount, long long base,
                                           long long pages, bool is_used) {
    int32_t c[kPlanItems];
#pragma unroll
    for (int i = 0; i < kPlanItems; ++i) {
        const long long p = tile_page(base, i);
        c[i] = p < pages ? refcount[p] : is_used ? 0 : 1;
    }
#pragma unroll
    for (int i = 0; i < kPlanItems; ++i) mask[i] = __ballot_sync(0xffffffffu, (c[i] > 0) == is_used);
}
// How many pages of the masks come before the warp's; `total` receives how many the tile has.
__device__ __forceinline__ int before_warp(const uint32_t (&mask)[kPlanItems], int *warps, int &total) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPlanItems; ++i) n += __popc(mask[i]);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();   // the last call's sums have been read
    if (lane == 0) warps[warp] = n;
    __syncthreads();
    const int w = warps[lane];
    total = __reduce_add_sync(0xffffffffu, w);
    return __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
}
__device__ __forceinline__ uint32_t lanes_before() { return (1u << (threadIdx.x & 31)) - 1; }

// Hands out the `want` lowest free pages: list[i] is the i-th, its count becomes 1.  Returns how many there were.
__device__ int take_free(int32_t *refcount, long long pages, long long want, int32_t *list, int *warps) {
    const int lane = threadIdx.x & 31;
    long long have = 0;
    for (long long base = 0; base < pages && have < want; base += kPlanTile) {
        uint32_t free_pages[kPlanItems];
        int total;
        load_masks(free_pages, refcount, base, pages, false);
        long long r = have + before_warp(free_pages, warps, total);
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i) {
            const long long at = r + __popc(free_pages[i] & lanes_before());
            if ((free_pages[i] >> lane & 1) && at < want) {
                const long long p = tile_page(base, i);
                list[at] = (int32_t)p;
                refcount[p] = 1;
            }
            r += __popc(free_pages[i]);
        }
        have += total;
    }
    return (int)(have < want ? have : want);
}

__device__ __forceinline__ long long clamp_length(int32_t len, long long width, int32_t page_tokens) {
    const long long top = width * page_tokens;
    return len < 0 ? 0 : len > top ? top : len;
}
__device__ __forceinline__ int32_t valid_page(int32_t p, long long pages) { return p >= 0 && p < pages ? p : -1; }

// One piece of one page of all pools' from page `from` to page `to`.
__device__ __forceinline__ void move_piece(const Pools &pools, int piece, long long from, long long to) {
    int k = 0;
    while (true) {   // at most PS_PAGES_MAX_POOLS steps
        const int of = (int)((pools.pool[k].page_bytes + kPiece - 1) / kPiece);
        if (piece < of) break;
        piece -= of;
        ++k;
    }
    const long long bytes = pools.pool[k].page_bytes, at = (long long)piece * kPiece;
    const int n = (int)min((long long)kPiece, bytes - at);
    const char *s = static_cast<const char *>(pools.pool[k].data) + from * bytes + at;
    char *d = static_cast<char *>(pools.pool[k].data) + to * bytes + at;
    if (((reinterpret_cast<uintptr_t>(s) | reinterpret_cast<uintptr_t>(d) | (uintptr_t)n) & 15) == 0) {
        constexpr int U = kPiece / 16 / kMoveThreads;
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = (u * kMoveThreads + (int)threadIdx.x) * 16;
            if (i < n) x[u] = __ldcs(reinterpret_cast<const uint4 *>(s + i));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = (u * kMoveThreads + (int)threadIdx.x) * 16;
            if (i < n) __stcs(reinterpret_cast<uint4 *>(d + i), x[u]);
        }
    } else {
        for (int i = threadIdx.x; i < n; i += kMoveThreads) d[i] = s[i];
    }
}

__global__ void __launch_bounds__(kMoveThreads) pages_copy_kernel(const Pools pools, long long pages, const int32_t *src,
                                                                  const int32_t *dst, long long n) {
    for (long long i = blockIdx.x; i < n * pools.pieces; i += gridDim.x) {
        const long long pair = i / pools.pieces;
        const int32_t s = valid_page(src[pair], pages), d = valid_page(dst[pair], pages);
        if (s >= 0 && d >= 0 && s != d) move_piece(pools, (int)(i % pools.pieces), s, d);
    }
}

// ---- fork -----------------------------------------------------------------------------

struct ForkArgs {
    const int32_t *table, *lengths, *parents;
    long long rows, width, new_rows, pages;
    int32_t page_tokens;
    int32_t *refcount, *new_table, *new_lengths, *missing;
    PlanSpace w;
};
// Row i's last page if it is part-filled (and to be copied), else -1.
__device__ __forceinline__ int32_t fork_page(const ForkArgs &a, long long i) {
    const int32_t p = a.parents[i];
    if (p < 0 || p >= a.rows) return -1;
    const long long len = clamp_length(a.lengths[p], a.width, a.page_tokens);
    return len % a.page_tokens ? valid_page(a.table[p * a.width + len / a.page_tokens], a.pages) : -1;
}
__global__ void __launch_bounds__(kPlanThreads) pages_fork_plan_kernel(const ForkArgs a) {
    __shared__ int warps[32];
    long long want = 0;
    for (long long base = 0; base < a.new_rows; base += kPlanThreads) {
        const long long i = base + threadIdx.x;
        const int need = i < a.new_rows && fork_page(a, i) >= 0;
        int total;
        const int r = block_exclusive(need, warps, total);
        if (i < a.new_rows) a.w.rank[i] = need ? (int32_t)(want + r) : -1;
        want += total;
    }
    const int have = take_free(a.refcount, a.pages, want, a.w.list, warps);
    if (threadIdx.x == 0) {
        a.w.head[0] = have;
        if (a.missing) *a.missing = (int32_t)(want - have);
    }
}
__global__ void __launch_bounds__(kMoveThreads) pages_fork_kernel(const ForkArgs a, const Pools pools) {
    const int have = a.w.head[0];
    const long long tasks = a.new_rows * (pools.pieces + 1);
    for (long long t = blockIdx.x; t < tasks; t += gridDim.x) {
        const long long i = t / (pools.pieces + 1);
        const int piece = (int)(t % (pools.pieces + 1));
        const int32_t rank = a.w.rank[i], to = rank >= 0 && rank < have ? a.w.list[rank] : -1;
        const int32_t p = a.parents[i];
        const bool ok = p >= 0 && p < a.rows;
        const long long len = ok ? clamp_length(a.lengths[p], a.width, a.page_tokens) : 0, full = len / a.page_tokens;
        if (piece < pools.pieces) {
            if (to >= 0) move_piece(pools, piece, a.table[p * a.width + full], to);
            continue;
        }
        for (long long j = threadIdx.x; j < a.width; j += kMoveThreads) {
            int32_t page = -1;
            if (j < full) {
                page = valid_page(a.table[p * a.width + j], a.pages);
                if (page >= 0) atomicAdd(a.refcount + page, 1);
            } else if (j == full) {
                page = to;
            }
            a.new_table[i * a.width + j] = page;
        }
        if (threadIdx.x == 0) a.new_lengths[i] = (int32_t)len;
    }
}

// ---- reorder --------------------------------------------------------------------------

struct ReorderArgs {
    const int32_t *slots, *parents;
    long long rows, pages;
    int32_t *new_slots, *missing;
    PlanSpace w;   // head[0]: pages to copy, rank[p]: the first row that continues row p, list: pages that no row continues
};
__device__ __forceinline__ int32_t reorder_parent(const ReorderArgs &a, long long i) {   // -1 for none that has a page
    const int32_t p = a.parents[i];
    return p >= 0 && p < a.rows && valid_page(a.slots[p], a.pages) >= 0 ? p : -1;
}
__global__ void __launch_bounds__(kPlanThreads) pages_reorder_plan_kernel(const ReorderArgs a) {
    __shared__ int warps[32];
    for (long long i = threadIdx.x; i < a.rows; i += kPlanThreads) a.w.rank[i] = INT_MAX;
    __syncthreads();
    for (long long i = threadIdx.x; i < a.rows; i += kPlanThreads) {
        const int32_t p = reorder_parent(a, i);
        if (p >= 0) atomicMin(a.w.rank + p, (int32_t)i);
    }
    __syncthreads();
    // pages that no row continues, and how many rows have to copy (a page named twice could make more of the first than pages)
    long long spare = 0, copies = 0;
    for (long long base = 0; base < a.rows; base += kPlanThreads) {
        const long long i = base + threadIdx.x;
        const bool in = i < a.rows;
        const int32_t page = in ? valid_page(a.slots[i], a.pages) : -1, p = in ? reorder_parent(a, i) : -1;
        const bool free_page = page >= 0 && __ldcg(a.w.rank + i) == INT_MAX;
        const bool copied = p >= 0 && __ldcg(a.w.rank + p) != i;
        int total;
        const long long at = spare + block_exclusive(free_page, warps, total);
        if (free_page && at < a.pages) a.w.list[at] = page;
        spare += total;
        block_exclusive(copied, warps, total);
        copies += total;
    }
    spare = min(spare, a.pages);
    __syncthreads();
    long long copy = 0, rest = copies;   // rows that copy come first, then those that continue none
    for (long long base = 0; base < a.rows; base += kPlanThreads) {
        const long long i = base + threadIdx.x;
        const bool in = i < a.rows;
        const int32_t p = in ? reorder_parent(a, i) : -1;
        const bool copied = p >= 0 && __ldcg(a.w.rank + p) != i, orphan = in && p < 0;
        int n_copied, n_orphan;
        const long long at_copy = copy + block_exclusive(copied, warps, n_copied);
        const long long at_rest = rest + block_exclusive(orphan, warps, n_orphan);
        if (in) {
            const long long at = copied ? at_copy : at_rest;
            const int32_t to = !copied && !orphan ? a.slots[p] : at < spare ? a.w.list[at] : -1;
            if (copied && to >= 0) {
                a.w.from[at] = a.slots[p];
                a.w.to[at] = to;
            }
            a.new_slots[i] = to;
        }
        copy += n_copied;
        rest += n_orphan;
    }
    if (threadIdx.x == 0) {
        a.w.head[0] = (int32_t)min(copies, spare);
        if (a.missing) *a.missing = (int32_t)max(copies - spare, 0ll);
    }
}
__global__ void __launch_bounds__(kMoveThreads) pages_reorder_kernel(const PlanSpace w, const Pools pools) {
    const long long tasks = (long long)w.head[0] * pools.pieces;
    for (long long t = blockIdx.x; t < tasks; t += gridDim.x) {
        const long long i = t / pools.pieces;
        move_piece(pools, (int)(t % pools.pieces), w.from[i], w.to[i]);
    }
}

// ---- grow -----------------------------------------------------------------------------

struct GrowArgs {
    int32_t *table;
    const int32_t *lengths, *new_lengths;
    long long rows, width, pages;
    int32_t page_tokens;
    int32_t *refcount, *missing;
    PlanSpace w;
};
__global__ void __launch_bounds__(kPlanThreads) pages_grow_kernel(const GrowArgs a) {
    __shared__ int warps[32];
    __shared__ unsigned long long past;
    if (threadIdx.x == 0) past = 0;
    // places of row r that are added and hold none, from `first` on; `beyond`: those past the width
    auto places = [&](long long r, long long &first, long long &last, long long &beyond) {
        const long long pt = a.page_tokens, len = clamp_length(a.lengths[r], a.width, a.page_tokens);
        const long long want = a.new_lengths[r] > 0 ? a.new_lengths[r] : 0;
        first = (len + pt - 1) / pt;
        last = (want + pt - 1) / pt;
        beyond = last > a.width ? last - max(first, a.width) : 0;
        if (last > a.width) last = a.width;
    };
    long long want = 0;
    __syncthreads();
    for (long long base = 0; base < a.rows; base += kPlanThreads) {
        const long long r = base + threadIdx.x;
        int need = 0, total;
        if (r < a.rows) {
            long long first, last, beyond;
            places(r, first, last, beyond);
            for (long long j = first; j < last; ++j) need += valid_page(a.table[r * a.width + j], a.pages) < 0;
            if (beyond > 0) atomicAdd(&past, (unsigned long long)beyond);
        }
        const int rank = block_exclusive(need, warps, total);
        if (r < a.rows) a.w.rank[r] = (int32_t)(want + rank);
        want += total;
    }
    const int have = take_free(a.refcount, a.pages, want, a.w.list, warps);
    __syncthreads();   // the list, written by all threads
    for (long long r = threadIdx.x; r < a.rows; r += kPlanThreads) {
        long long first, last, beyond;
        places(r, first, last, beyond);
        int rank = a.w.rank[r];
        for (long long j = first; j < last; ++j) {
            int32_t *at = a.table + r * a.width + j;
            if (valid_page(*at, a.pages) < 0) {
                *at = rank < have ? a.w.list[rank] : -1;
                ++rank;
            }
        }
    }
    if (threadIdx.x == 0 && a.missing) *a.missing = (int32_t)min(want - have + (long long)past, (long long)INT_MAX);
}

// ---- free -----------------------------------------------------------------------------

__global__ void __launch_bounds__(kMoveThreads) pages_free_kernel(int32_t *table, long long rows, long long width,
                                                                  const uint8_t *flags, int32_t *refcount, long long pages) {
    const long long n = rows * width;
    for (long long i = (long long)blockIdx.x * kMoveThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kMoveThreads) {
        if (flags && flags[i / width] == 0) continue;
        const int32_t p = valid_page(table[i], pages);
        if (p >= 0) atomicSub(refcount + p, 1);
        table[i] = -1;
    }
}

// ---- compact --------------------------------------------------------------------------

struct CompactArgs {
    int32_t *table;
    long long rows, width, pages;
    int32_t *refcount, *used;
    PlanSpace w;   // head[0]: pages to move, list: the free pages below m, from: the used ones from m on,
                   // to[p]: p where page p stays, -1 where it is free, -2 - i for the i-th one that moves
};
__global__ void __launch_bounds__(kPlanThreads) pages_compact_plan_kernel(const CompactArgs a) {
    __shared__ int warps[32];
    __shared__ int below;   // pages in use below m
    const int lane = threadIdx.x & 31;
    uint32_t used[kPlanItems];
    long long m = 0;
    for (long long base = 0; base < a.pages; base += kPlanTile) {
        int total;
        load_masks(used, a.refcount, base, a.pages, true);
        before_warp(used, warps, total);
        m += total;
    }
    if (threadIdx.x == 0) below = (int)m;   // m == pages: nothing moves
    long long rank = 0;                     // pages in use before the tile
    for (long long base = 0; base < a.pages; base += kPlanTile) {
        int total;
        if (a.pages > kPlanTile) load_masks(used, a.refcount, base, a.pages, true);
        const long long r0 = rank + before_warp(used, warps, total);
        long long r = r0;
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i) {
            if (tile_page(base, i) == m && m < a.pages) below = (int)(r + __popc(used[i] & lanes_before()));
            r += __popc(used[i]);
        }
        __syncthreads();
        r = r0;
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i) {
            const long long p = tile_page(base, i), at = r + __popc(used[i] & lanes_before());
            if (p < a.pages) {
                const bool in = used[i] >> lane & 1;
                if (in && p >= m) a.w.from[at - below] = (int32_t)p;
                if (!in && p < m) a.w.list[p - at] = (int32_t)p;
                a.w.to[p] = !in ? -1 : p < m ? (int32_t)p : -2 - (int32_t)(at - below);
            }
            r += __popc(used[i]);
        }
        rank += total;
    }
    __syncthreads();
    const int moves = (int)(m - below);
    if (threadIdx.x == 0) {
        a.w.head[0] = moves;
        if (a.used) *a.used = (int32_t)m;
    }
}
__global__ void __launch_bounds__(kMoveThreads) pages_compact_kernel(const CompactArgs a, const Pools pools) {
    const long long tasks = (long long)a.w.head[0] * pools.pieces;
    for (long long t = blockIdx.x; t < tasks; t += gridDim.x) {
        const long long i = t / pools.pieces;
        move_piece(pools, (int)(t % pools.pieces), a.w.from[i], a.w.list[i]);
    }
    for (long long i = (long long)blockIdx.x * kMoveThreads + threadIdx.x; i < a.w.head[0]; i += (long long)gridDim.x * kMoveThreads) {
        const int32_t f = a.w.from[i], to = a.w.list[i];   // no page is on both lists
        a.refcount[to] = a.refcount[f];
        a.refcount[f] = 0;
    }
    const long long n = a.rows * a.width;
    for (long long i = (long long)blockIdx.x * kMoveThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kMoveThreads) {
        const int32_t p = valid_page(a.table[i], a.pages);
        const int32_t to = p >= 0 ? a.w.to[p] : -1;
        a.table[i] = to >= -1 ? to : a.w.list[-2 - to];
    }
}

// ---- host -----------------------------------------------------------------------------

struct Bytes {
    uintptr_t a, b;
};
Bytes bytes_of(const void *p, size_t n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, p ? a + n : a};
}
bool meet(const Bytes &x, const Bytes &y) { return x.a < y.b && y.a < x.b; }

ps_status done(cudaError_t e) {
    if (e == cudaSuccess) return PS_OK;
    note_cuda_error(e);
    return PS_ERR_CUDA;
}
bool aligned4(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }
bool sizes_ok(long long rows, long long width, long long pages) {
    return rows >= 0 && width >= 0 && pages >= 0 && rows <= INT_MAX && width <= INT_MAX && pages <= INT_MAX &&
           (width == 0 || rows <= INT_MAX / width);
}
ps_status pools_of(const ps_page_pool *pools, int n, long long pages, Pools &out) {
    if (n < 0 || n > PS_PAGES_MAX_POOLS || (n > 0 && pools == nullptr)) return PS_ERR_INVALID_ARG;
    out.n = n;
    long long pieces = 0;
    for (int i = 0; i < n; ++i) {
        if (pools[i].page_bytes < 1 || pools[i].page_bytes > (1ll << 40)) return PS_ERR_INVALID_ARG;
        if (pools[i].data == nullptr && pages > 0) return PS_ERR_INVALID_ARG;
        out.pool[i] = pools[i];
        pieces += (pools[i].page_bytes + kPiece - 1) / kPiece;
        for (int j = 0; j < i; ++j)
            if (meet(bytes_of(pools[i].data, (size_t)(pages * pools[i].page_bytes)),
                     bytes_of(pools[j].data, (size_t)(pages * pools[j].page_bytes))))
                return PS_ERR_OVERLAP;
    }
    if (pieces > INT_MAX) return PS_ERR_INVALID_ARG;
    out.pieces = (int)pieces;
    return PS_OK;
}
// No array of `list` may meet another, or a pool.
template <int N>
bool arrays_meet(const Bytes (&list)[N], const Pools &pools, long long pages) {
    for (int i = 0; i < N; ++i) {
        for (int j = i + 1; j < N; ++j)
            if (meet(list[i], list[j])) return true;
        for (int k = 0; k < pools.n; ++k)
            if (meet(list[i], bytes_of(pools.pool[k].data, (size_t)(pages * pools.pool[k].page_bytes)))) return true;
    }
    return false;
}
unsigned move_grid(long long tasks) { return (unsigned)(tasks < 1 ? 1 : tasks < kMoveCtas ? tasks : kMoveCtas); }

}  // namespace

}  // namespace ps

using namespace ps;

extern "C" size_t ps_pages_workspace_size(int64_t rows, int64_t pages) {
    if (!sizes_ok(rows, 1, pages)) return 0;
    return 4 * (64 + ints((size_t)rows) + 3 * ints((size_t)pages));
}

extern "C" ps_status ps_pages_copy(const ps_page_pool *pools, int npools, int64_t pages, const int32_t *src,
                                   const int32_t *dst, int64_t n, ps_stream_t stream) {
    Pools p{};
    if (!sizes_ok(n, 1, pages)) return PS_ERR_INVALID_ARG;
    const ps_status st = pools_of(pools, npools, pages, p);
    if (st != PS_OK) return st;
    if (n == 0 || pages == 0 || npools == 0) return PS_OK;
    if (src == nullptr || dst == nullptr || !aligned4(src) || !aligned4(dst)) return PS_ERR_INVALID_ARG;
    for (int k = 0; k < npools; ++k) {
        const Bytes b = bytes_of(p.pool[k].data, (size_t)(pages * p.pool[k].page_bytes));
        if (meet(b, bytes_of(src, (size_t)n * 4)) || meet(b, bytes_of(dst, (size_t)n * 4))) return PS_ERR_OVERLAP;
    }
    pages_copy_kernel<<<move_grid(n * p.pieces), kMoveThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p, pages, src, dst, n);
    return done(cudaGetLastError());
}

extern "C" ps_status ps_pages_fork(const int32_t *table, const int32_t *lengths, int64_t rows, int64_t width,
                                   const int32_t *parents, int64_t new_rows, int32_t page_tokens, int32_t *refcount,
                                   const ps_page_pool *pools, int npools, int64_t pages, int32_t *new_table,
                                   int32_t *new_lengths, int32_t *missing, void *ws, size_t ws_bytes, ps_stream_t stream) {
    Pools p{};
    if (!sizes_ok(rows, width, pages) || !sizes_ok(new_rows, width, pages) || page_tokens < 1) return PS_ERR_INVALID_ARG;
    const ps_status st = pools_of(pools, npools, pages, p);
    if (st != PS_OK) return st;
    if (!aligned4(table) || !aligned4(lengths) || !aligned4(parents) || !aligned4(refcount) || !aligned4(new_table) ||
        !aligned4(new_lengths) || !aligned4(missing) || reinterpret_cast<uintptr_t>(ws) % 256 != 0)
        return PS_ERR_INVALID_ARG;
    if ((rows > 0 && (lengths == nullptr || (table == nullptr && width > 0))) || (pages > 0 && refcount == nullptr) ||
        (new_rows > 0 && (parents == nullptr || new_lengths == nullptr || (new_table == nullptr && width > 0))) || ws == nullptr)
        return PS_ERR_INVALID_ARG;
    const size_t need = ps_pages_workspace_size(new_rows, pages);
    if (ws_bytes < need) return PS_ERR_WORKSPACE_TOO_SMALL;
    const Bytes list[] = {bytes_of(table, (size_t)(rows * width) * 4), bytes_of(lengths, (size_t)rows * 4),
                          bytes_of(parents, (size_t)new_rows * 4), bytes_of(refcount, (size_t)pages * 4),
                          bytes_of(new_table, (size_t)(new_rows * width) * 4), bytes_of(new_lengths, (size_t)new_rows * 4),
                          bytes_of(missing, 4), bytes_of(ws, need)};
    if (arrays_meet(list, p, pages)) return PS_ERR_OVERLAP;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const ForkArgs a{table, lengths, parents, rows, width, new_rows, pages, page_tokens, refcount, new_table, new_lengths,
                     missing, plan_space(ws, new_rows, pages)};
    pages_fork_plan_kernel<<<1, kPlanThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && new_rows > 0) {
        pages_fork_kernel<<<move_grid(new_rows * (p.pieces + 1)), kMoveThreads, 0, s>>>(a, p);
        e = cudaGetLastError();
    }
    return done(e);
}

extern "C" ps_status ps_pages_reorder(const int32_t *slots, const int32_t *parents, int64_t rows, const ps_page_pool *pools,
                                      int npools, int64_t pages, int32_t *new_slots, int32_t *missing, void *ws, size_t ws_bytes,
                                      ps_stream_t stream) {
    Pools p{};
    if (!sizes_ok(rows, 1, pages)) return PS_ERR_INVALID_ARG;
    const ps_status st = pools_of(pools, npools, pages, p);
    if (st != PS_OK) return st;
    if (!aligned4(slots) || !aligned4(parents) || !aligned4(new_slots) || !aligned4(missing) || reinterpret_cast<uintptr_t>(ws) % 256 != 0)
        return PS_ERR_INVALID_ARG;
    if ((rows > 0 && (slots == nullptr || parents == nullptr || new_slots == nullptr)) || ws == nullptr) return PS_ERR_INVALID_ARG;
    const size_t need = ps_pages_workspace_size(rows, pages);
    if (ws_bytes < need) return PS_ERR_WORKSPACE_TOO_SMALL;
    const Bytes list[] = {bytes_of(slots, (size_t)rows * 4), bytes_of(parents, (size_t)rows * 4), bytes_of(new_slots, (size_t)rows * 4),
                          bytes_of(missing, 4), bytes_of(ws, need)};
    if (arrays_meet(list, p, pages)) return PS_ERR_OVERLAP;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const ReorderArgs a{slots, parents, rows, pages, new_slots, missing, plan_space(ws, rows, pages)};
    pages_reorder_plan_kernel<<<1, kPlanThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && rows > 1 && p.pieces > 0) {   // at least one row keeps its page or has none
        pages_reorder_kernel<<<move_grid((rows < pages ? rows : pages) * p.pieces), kMoveThreads, 0, s>>>(a.w, p);
        e = cudaGetLastError();
    }
    return done(e);
}

extern "C" ps_status ps_pages_grow(int32_t *table, const int32_t *lengths, const int32_t *new_lengths, int64_t rows,
                                   int64_t width, int32_t page_tokens, int32_t *refcount, int64_t pages, int32_t *missing,
                                   void *ws, size_t ws_bytes, ps_stream_t stream) {
    if (!sizes_ok(rows, width, pages) || page_tokens < 1) return PS_ERR_INVALID_ARG;
    if (!aligned4(table) || !aligned4(lengths) || !aligned4(new_lengths) || !aligned4(refcount) || !aligned4(missing) ||
        reinterpret_cast<uintptr_t>(ws) % 256 != 0)
        return PS_ERR_INVALID_ARG;
    if ((rows > 0 && (lengths == nullptr || new_lengths == nullptr || (table == nullptr && width > 0))) ||
        (pages > 0 && refcount == nullptr) || ws == nullptr)
        return PS_ERR_INVALID_ARG;
    const size_t need = ps_pages_workspace_size(rows, pages);
    if (ws_bytes < need) return PS_ERR_WORKSPACE_TOO_SMALL;
    const Bytes list[] = {bytes_of(table, (size_t)(rows * width) * 4), bytes_of(new_lengths, (size_t)rows * 4),
                          bytes_of(refcount, (size_t)pages * 4), bytes_of(missing, 4), bytes_of(ws, need),
                          bytes_of(lengths == new_lengths ? nullptr : lengths, (size_t)rows * 4)};
    if (arrays_meet(list, Pools{}, 0)) return PS_ERR_OVERLAP;
    const GrowArgs a{table, lengths, new_lengths, rows, width, pages, page_tokens, refcount, missing, plan_space(ws, rows, pages)};
    pages_grow_kernel<<<1, kPlanThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    return done(cudaGetLastError());
}

extern "C" ps_status ps_pages_free(int32_t *table, int64_t rows, int64_t width, const uint8_t *flags, int32_t *refcount,
                                   int64_t pages, ps_stream_t stream) {
    if (!sizes_ok(rows, width, pages)) return PS_ERR_INVALID_ARG;
    if (rows * width == 0) return PS_OK;
    if (table == nullptr || !aligned4(table) || (pages > 0 && refcount == nullptr) || !aligned4(refcount)) return PS_ERR_INVALID_ARG;
    const Bytes list[] = {bytes_of(table, (size_t)(rows * width) * 4), bytes_of(refcount, (size_t)pages * 4),
                          bytes_of(flags, (size_t)rows)};
    if (arrays_meet(list, Pools{}, 0)) return PS_ERR_OVERLAP;
    pages_free_kernel<<<move_grid((rows * width + kMoveThreads - 1) / kMoveThreads), kMoveThreads, 0,
                        reinterpret_cast<cudaStream_t>(stream)>>>(table, rows, width, flags, refcount, pages);
    return done(cudaGetLastError());
}

extern "C" ps_status ps_pages_compact(int32_t *table, int64_t rows, int64_t width, int32_t *refcount,
                                      const ps_page_pool *pools, int npools, int64_t pages, int32_t *used, void *ws,
                                      size_t ws_bytes, ps_stream_t stream) {
    Pools p{};
    if (!sizes_ok(rows, width, pages)) return PS_ERR_INVALID_ARG;
    const ps_status st = pools_of(pools, npools, pages, p);
    if (st != PS_OK) return st;
    if (!aligned4(table) || !aligned4(refcount) || !aligned4(used) || reinterpret_cast<uintptr_t>(ws) % 256 != 0)
        return PS_ERR_INVALID_ARG;
    if ((rows * width > 0 && table == nullptr) || (pages > 0 && refcount == nullptr) || ws == nullptr) return PS_ERR_INVALID_ARG;
    const size_t need = ps_pages_workspace_size(0, pages);
    if (ws_bytes < need) return PS_ERR_WORKSPACE_TOO_SMALL;
    const Bytes list[] = {bytes_of(table, (size_t)(rows * width) * 4), bytes_of(refcount, (size_t)pages * 4), bytes_of(used, 4),
                          bytes_of(ws, need)};
    if (arrays_meet(list, p, pages)) return PS_ERR_OVERLAP;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const CompactArgs a{table, rows, width, pages, refcount, used, plan_space(ws, 0, pages)};
    pages_compact_plan_kernel<<<1, kPlanThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && pages > 0) {
        const long long tasks = (long long)p.pieces * pages / 2 + (rows * width + pages / 2) / kMoveThreads + 1;
        pages_compact_kernel<<<move_grid(tasks), kMoveThreads, 0, s>>>(a, p);
        e = cudaGetLastError();
    }
    return done(e);
}
