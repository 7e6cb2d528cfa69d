// pages.cu -- the pages of a paged cache, managed on the device: rows of the
// block table share pages (fork), grow (extend, copying a shared partial page
// before it is written), shrink or end (free), and the pool is compacted.
//
// The only state beside the block table and seq_lens is refcount [NP]: page p
// is free when refcount[p] == 0.  New pages are the lowest free ids, in the
// order of the call's rows, so the result depends on nothing but the inputs:
// there is no free list whose order could, and refcounts change by integer
// atomics only.
//
// "The k-th free page" is a prefix count over refcount, in tiles of 4096 pages, one
// CTA each.  For pools of up to kDirectTiles tiles every CTA sums the tiles before
// its own itself (from L2); larger ones count the tiles in a launch before.  The
// free pages are listed by rank, a first CTA prefix-sums what each row needs, and
// the next launch takes each row's pages from that list, copies page data and
// publishes lengths.  Each launch overlaps the end of the one before.
//
// Measured: 28 forks of 4 rows and the growth of all 32 by a token, 32 shared pages of
// 256 KiB copied, 12 us with the copies of the tables (17 MB); 85 of 256 rows freed
// and 33 k pages of 4 KiB compacted, 25 us with the same, 12 us of it the move of 7.7 k
// pages (63 MB, 0.78 of the copy rate).  The rest is the latency of dependent loads
// and launches.
#include "common.cuh"
#include "internal.h"

namespace aq {

namespace {

constexpr int kThreads = 1024;
constexpr int kTile = 4 * kThreads;
constexpr int kMaxPools = 256;
// Pools of up to 6 tiles are counted without a launch of its own.  An extend without /
// with it, us: 4.1 / 5.6 at 1 tile, 5.6 / 6.2 at 6, 7.5 / 6.3 at 16; a compaction: 5.2 /
// 6.8, 6.9 / 6.8, 9.1 / 7.0.
constexpr int kDirectTiles = 6;
constexpr int kCopyThreads = 256;

struct PageParams {
    int32_t *block_table;          // [R][max_pages]
    int32_t *seq_lens;             // [R]
    int32_t *refcount;             // [NP]
    const int32_t *rows, *args;    // [n]: extend: rows, new lengths; fork: sources, destinations; free: rows, kept lengths
    int32_t *status;
    // workspace
    int32_t *tiles;                // [ntiles] pages counted per tile
    int32_t *total;                // [4]: free or live pages, movers
    long long *off;                // [R + 1] prefix of the rows' needs
    int32_t *info;                 // [R]
    int32_t *claim;                // [R]
    int32_t *from;                 // [R] shared partial page to copy, or -1
    int32_t *rank, *movers, *holes;    // [NP]; movers: an extend's free pages by rank
    int32_t n, num_rows, max_pages, num_pages, ntiles;
};

// The pools, cut into chunks of kChunk bytes: those of pool k are first[k] ..
// first[k + 1] - 1.  A warp copies one chunk of one page at a time.
constexpr int kChunk = 4096;
struct PagePools {
    aq_page_pool pool[kMaxPools];
    int32_t first[kMaxPools + 1];
    int32_t n;
};

// Exclusive prefix of `v` over the block; *sum = the block's total.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *sum) {
    __shared__ T part[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const T y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();                                   // part of an earlier call has been read
    if (lane == 31) part[warp] = x;
    __syncthreads();
    if (warp == 0) {
        T y = part[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const T z = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) y += z;
        }
        part[lane] = y;
    }
    __syncthreads();
    *sum = part[kThreads / 32 - 1];
    return x - v + (warp ? part[warp - 1] : 0);
}

__device__ __forceinline__ bool row_ok(const PageParams &p, int row) { return row >= 0 && row < p.num_rows; }

__device__ __forceinline__ bool len_ok(const PageParams &p, int len) {
    return len >= 0 && len <= static_cast<int64_t>(p.max_pages) * kPage;
}

// The first of the call's entries that names a row owns it: claim[row] = the
// lowest index.  Called by one CTA; entries outside [0, R) are left out.
__device__ __forceinline__ void claim_rows(const PageParams &p, const int32_t *rows) {
    for (int i = threadIdx.x; i < p.n; i += kThreads)
        if (row_ok(p, rows[i])) p.claim[rows[i]] = 0x7fffffff;
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += kThreads)
        if (row_ok(p, rows[i])) atomicMin(&p.claim[rows[i]], i);
    __syncthreads();
}

// Pages of tile `t`, four per thread; those outside the pool count as neither
// free nor live (-1).
__device__ __forceinline__ int4 tile_counts(const PageParams &p, int t) {
    const int64_t i = static_cast<int64_t>(t) * kTile + 4 * threadIdx.x;
    int4 r = make_int4(-1, -1, -1, -1);
    if (i + 4 <= p.num_pages) r = *reinterpret_cast<const int4 *>(p.refcount + i);
    else {
        if (i < p.num_pages) r.x = p.refcount[i];
        if (i + 1 < p.num_pages) r.y = p.refcount[i + 1];
        if (i + 2 < p.num_pages) r.z = p.refcount[i + 2];
    }
    return r;
}

// What row entry i of an extend needs; info[i] = 1: its shared partial page is
// copied first, -1: a data error, the row stays as it is.
__device__ __forceinline__ int extend_need(const PageParams &p, int i) {
    p.info[i] = -1;
    p.from[i] = -1;
    const int row = p.rows[i], len = p.args[i];
    if (!row_ok(p, row) || __ldcg(&p.claim[row]) != i) {
        flag_status(p.status, AQ_DEV_BAD_ROW);
        return 0;
    }
    const int L = p.seq_lens[row];
    if (!len_ok(p, L) || !len_ok(p, len) || len < L) {
        flag_status(p.status, AQ_DEV_BAD_LENGTH);
        return 0;
    }
    const int have = (L + kPage - 1) / kPage, want = (len - 1) / kPage + 1;
    int copy = 0;
    if (len > L && L % kPage) {
        const int pg = p.block_table[static_cast<size_t>(row) * p.max_pages + have - 1];
        if (pg < 0 || pg >= p.num_pages) {
            flag_status(p.status, AQ_DEV_BAD_PAGE);
            return 0;
        }
        copy = p.refcount[pg] > 1;
        if (copy) p.from[i] = pg;
    }
    p.info[i] = copy;
    return len > L ? want - have + copy : 0;
}

__device__ __forceinline__ void begin() {
    grid_dependency_wait();
    grid_launch_dependents();
}

// The page counts of the tiles: free pages (FREE) or live ones.
template <bool FREE>
__device__ __forceinline__ int count4(const int4 &r) {
    return FREE ? (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0) : (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
}

template <bool FREE>
__global__ void __launch_bounds__(kThreads) pages_count_kernel(const __grid_constant__ PageParams p) {
    begin();
    int sum;
    block_scan(count4<FREE>(tile_counts(p, blockIdx.x)), &sum);
    if (threadIdx.x == 0) p.tiles[blockIdx.x] = sum;
}

// The pages counted in tiles before `t`, and in all of them (one scan of both).
template <bool FREE>
__device__ __forceinline__ int tiles_before(const PageParams &p, int t, int *total) {
    unsigned long long both = 0, sum;
    if (p.ntiles <= kDirectTiles) {
#pragma unroll 4
        for (int i = 0; i < p.ntiles; ++i) {
            const unsigned long long x = static_cast<unsigned>(count4<FREE>(tile_counts(p, i)));
            both += (x << 32) + (i < t ? x : 0u);
        }
    } else {
        for (int i = threadIdx.x; i < p.ntiles; i += kThreads) {
            const unsigned long long x = static_cast<unsigned>(p.tiles[i]);
            both += (x << 32) + (i < t ? x : 0u);
        }
    }
    block_scan(both, &sum);
    *total = static_cast<int>(sum >> 32);
    return static_cast<int>(sum & 0xffffffffu);
}

// An extend's free pages by rank (CTAs 1 on, a tile each) and the rows' needs with
// their prefix (CTA 0).
__global__ void __launch_bounds__(kThreads) pages_assign_kernel(const __grid_constant__ PageParams p) {
    begin();
    if (blockIdx.x == 0) {
        claim_rows(p, p.rows);
        long long base = 0;
        for (int i0 = 0; i0 < p.n; i0 += kThreads) {
            const int i = i0 + threadIdx.x;
            long long sum;
            const long long need = i < p.n ? extend_need(p, i) : 0;
            const long long at = block_scan(need, &sum);
            if (i < p.n) p.off[i] = base + at;
            base += sum;
        }
        if (threadIdx.x == 0) p.off[p.n] = base;
        return;
    }
    const int t = blockIdx.x - 1;
    const int4 r = tile_counts(p, t);
    int total, sum;
    const int base = tiles_before<true>(p, t, &total);
    if (t == 0 && threadIdx.x == 0) p.total[0] = total;
    int rank = base + block_scan(count4<true>(r), &sum);
    const int f[4] = {r.x == 0, r.y == 0, r.z == 0, r.w == 0};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (f[k]) p.movers[rank++] = t * kTile + 4 * threadIdx.x + k;
}

// Chunk c of page `from` to page `to`, by one warp: up to 8 loads of 16 bytes per
// lane under way.  Pages that are no multiple of 16 bytes move by words.
__device__ __forceinline__ void copy_chunk(const PagePools &pools, int64_t from, int64_t to, int c, int lane) {
    int lo = 0, hi = pools.n;                          // the pool of chunk c
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (pools.first[mid] <= c) lo = mid;
        else hi = mid;
    }
    const int64_t bytes = pools.pool[lo].page_bytes, at = static_cast<int64_t>(c - pools.first[lo]) * kChunk;
    const int n = static_cast<int>(min(bytes - at, static_cast<int64_t>(kChunk)));
    unsigned char *data = static_cast<unsigned char *>(pools.pool[lo].data);
    const unsigned char *src = data + from * bytes + at;
    unsigned char *dst = data + to * bytes + at;
    if (bytes % 16 == 0) {
        uint4 x[kChunk / 512];
#pragma unroll
        for (int j = 0; j < kChunk / 512; ++j)
            if (512 * j + 16 * lane < n) x[j] = ld_global_na_v4(src + 512 * j + 16 * lane);
#pragma unroll
        for (int j = 0; j < kChunk / 512; ++j)
            if (512 * j + 16 * lane < n) *reinterpret_cast<uint4 *>(dst + 512 * j + 16 * lane) = x[j];
    } else {
        for (int i = 4 * lane; i < n; i += 128)
            *reinterpret_cast<uint32_t *>(dst + i) = *reinterpret_cast<const uint32_t *>(src + i);
    }
}

// Last launch of an extend, CTAs (row entry, part): the row's new table entries,
// its reference to a shared partial page dropped and the page copied, its length
// published.
__global__ void __launch_bounds__(kCopyThreads) pages_grow_kernel(const __grid_constant__ PageParams p,
                                                                  const __grid_constant__ PagePools pools) {
    begin();
    const int i = blockIdx.x, copy = p.info[i];
    if (copy < 0) return;
    const long long at = p.off[i], end = p.off[i + 1];
    if (end > (p.ntiles ? p.total[0] : 0) && end > at) {                // (a row that needs no page is served in any case)
        if (blockIdx.y == 0 && threadIdx.x == 0) flag_status(p.status, AQ_DEV_NO_PAGE);
        return;
    }
    const int from = p.from[i];
    if (blockIdx.y == 0) {
        const int row = p.rows[i], len = p.args[i], want = (len + kPage - 1) / kPage;
        const int first = want - static_cast<int>(end - at);               // the copied page's entry among them
        int32_t *bt = p.block_table + static_cast<size_t>(row) * p.max_pages;
        for (int j = threadIdx.x; j < want - first; j += kCopyThreads) {
            const int pg = p.movers[at + j];
            bt[first + j] = pg;
            p.refcount[pg] = 1;
        }
        if (threadIdx.x == 0) {
            p.seq_lens[row] = len;
            if (copy) atomicSub(&p.refcount[from], 1);
        }
    }
    if (!copy) return;
    const int to = p.movers[at], chunks = pools.first[pools.n];
    for (int c = blockIdx.y * (kCopyThreads / 32) + threadIdx.x / 32; c < chunks; c += gridDim.y * (kCopyThreads / 32))
        copy_chunk(pools, from, to, c, threadIdx.x & 31);
}

// Fork, a CTA per entry.  An entry whose destination is named before, or whose source
// is a destination, is refused: no row is then both read and written.
__global__ void __launch_bounds__(kThreads) pages_fork_kernel(const __grid_constant__ PageParams p) {
    begin();
    const int i = blockIdx.x, src = p.rows[i], dst = p.args[i];
    bool clash = false;
    for (int j = threadIdx.x; j < p.n; j += kThreads) {
        const int d = p.args[j];
        clash |= d == src || (j < i && d == dst);
    }
    __shared__ int len;
    if (threadIdx.x == 0) {
        len = -1;
        if (!row_ok(p, src) || !row_ok(p, dst) || p.seq_lens[dst] != 0) flag_status(p.status, AQ_DEV_BAD_ROW);
        else if (!len_ok(p, p.seq_lens[src])) flag_status(p.status, AQ_DEV_BAD_LENGTH);
        else len = p.seq_lens[src];
    }
    if (__syncthreads_or(clash)) {
        if (threadIdx.x == 0) flag_status(p.status, AQ_DEV_BAD_ROW);
        return;
    }
    const int L = len, n = (L + kPage - 1) / kPage;
    if (L < 0) return;
    const int32_t *from = p.block_table + static_cast<size_t>(src) * p.max_pages;
    int32_t *to = p.block_table + static_cast<size_t>(dst) * p.max_pages;
    for (int j = threadIdx.x; j < n; j += kThreads) {
        const int pg = from[j];
        to[j] = pg;
        if (pg < 0 || pg >= p.num_pages || atomicAdd(&p.refcount[pg], 1) <= 0) flag_status(p.status, AQ_DEV_BAD_PAGE);
    }
    if (threadIdx.x == 0) p.seq_lens[dst] = L;
}

// Free: a row keeps its first `keep` tokens.  The atomic minimum makes a row
// named twice lose each page once, whichever entry comes first.
__global__ void __launch_bounds__(kCopyThreads) pages_free_kernel(const __grid_constant__ PageParams p) {
    __shared__ int len;
    begin();
    const int row = p.rows[blockIdx.x], keep = p.args ? p.args[blockIdx.x] : 0;
    if (threadIdx.x == 0) {
        len = 0;
        if (!row_ok(p, row)) flag_status(p.status, AQ_DEV_BAD_ROW);
        else if (keep < 0 || !len_ok(p, *static_cast<volatile int32_t *>(p.seq_lens + row)))
            flag_status(p.status, AQ_DEV_BAD_LENGTH);
        else len = atomicMin(&p.seq_lens[row], keep);
    }
    __syncthreads();
    const int n = (len + kPage - 1) / kPage;
    for (int j = (max(keep, 0) + kPage - 1) / kPage + threadIdx.x; j < n; j += kCopyThreads) {
        int32_t *e = p.block_table + static_cast<size_t>(row) * p.max_pages + j;
        const int pg = *e;
        *e = -1;
        if (pg < 0 || pg >= p.num_pages) flag_status(p.status, AQ_DEV_BAD_PAGE);
        else if (atomicSub(&p.refcount[pg], 1) <= 0) {
            atomicAdd(&p.refcount[pg], 1);
            flag_status(p.status, AQ_DEV_BAD_PAGE);
        }
    }
}

// Second launch of a compaction: with N live pages, live page p >= N is the
// mover of rank (live pages in [N, p)), free page p < N the hole of rank (free
// pages in [0, p)); there are as many movers as holes.
__global__ void __launch_bounds__(kThreads) pages_map_kernel(const __grid_constant__ PageParams p) {
    begin();
    const int4 r = tile_counts(p, blockIdx.x);
    int live;
    const int base = tiles_before<false>(p, blockIdx.x, &live);
    // live pages below N: whole tiles, and the part of the tile that holds N
    const int cut = live / kTile;
    int under = 0;
    if (cut < p.ntiles) {
        const int4 s = tile_counts(p, cut);
        const int i = cut * kTile + 4 * threadIdx.x;
        int n = (s.x > 0 && i < live) + (s.y > 0 && i + 1 < live) + (s.z > 0 && i + 2 < live) + (s.w > 0 && i + 3 < live);
        if (p.ntiles <= kDirectTiles) {
            for (int t = 0; t < cut; ++t) n += count4<false>(tile_counts(p, t));
        } else {
            for (int t = threadIdx.x; t < cut; t += kThreads) n += p.tiles[t];
        }
        block_scan(n, &under);
    } else {
        under = live;                                  // every page is live
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.total[0] = live;
        p.total[1] = live - under;
    }
    const int c[4] = {r.x, r.y, r.z, r.w};
    int sum;
    int before = base + block_scan((c[0] > 0) + (c[1] > 0) + (c[2] > 0) + (c[3] > 0), &sum);
    for (int k = 0; k < 4; ++k) {
        const int64_t pg = static_cast<int64_t>(blockIdx.x) * kTile + 4 * threadIdx.x + k;
        if (pg >= p.num_pages) return;
        int rank = -1;
        if (c[k] > 0) {
            if (pg >= live) {
                rank = before - under;
                p.movers[rank] = static_cast<int>(pg);
            }
            ++before;
        } else if (pg < live) {
            p.holes[pg - before] = static_cast<int>(pg);
        }
        p.rank[pg] = rank;
    }
}

// Last launch of a compaction: movers are copied into holes and the block
// table rewritten (the first `table_ctas` CTAs).
__global__ void __launch_bounds__(kCopyThreads) pages_move_kernel(const __grid_constant__ PageParams p,
                                                                  const __grid_constant__ PagePools pools,
                                                                  int table_ctas) {
    begin();
    const int live = p.total[0], moves = p.total[1];
    if (static_cast<int>(blockIdx.x) < table_ctas) {
        for (int row = blockIdx.x; row < p.num_rows; row += table_ctas) {
            const int L = p.seq_lens[row];
            if (!len_ok(p, L)) {
                if (threadIdx.x == 0) flag_status(p.status, AQ_DEV_BAD_LENGTH);
                continue;
            }
            int32_t *bt = p.block_table + static_cast<size_t>(row) * p.max_pages;
            for (int j = threadIdx.x; j < (L + kPage - 1) / kPage; j += kCopyThreads) {
                const int pg = bt[j];
                if (pg >= 0 && pg < live) continue;
                const int rank = pg >= 0 && pg < p.num_pages ? p.rank[pg] : -1;
                if (rank < 0) flag_status(p.status, AQ_DEV_BAD_PAGE);
                else bt[j] = p.holes[rank];
            }
        }
        return;
    }
    const int chunks = pools.first[pools.n], lane = threadIdx.x & 31;
    const int64_t w0 = static_cast<int64_t>(blockIdx.x - table_ctas) * (kCopyThreads / 32) + threadIdx.x / 32;
    const int64_t nw = static_cast<int64_t>(gridDim.x - table_ctas) * (kCopyThreads / 32);
    for (int64_t i = w0 * 32 + lane; i < moves; i += nw * 32) {
        const int from = p.movers[i];
        p.refcount[p.holes[i]] = p.refcount[from];
        p.refcount[from] = 0;
    }
    for (int64_t u = w0; u < static_cast<int64_t>(moves) * chunks; u += nw) {
        const int64_t i = u / chunks;
        copy_chunk(pools, p.movers[i], p.holes[i], static_cast<int>(u % chunks), lane);
    }
}

bool off16(const void *a) { return (reinterpret_cast<uintptr_t>(a) & 15u) != 0; }

int tiles_of(int64_t pages) { return static_cast<int>((pages + kTile - 1) / kTile); }

// Workspace: int32 arrays in this order, each from a 16-byte boundary.
size_t ints(int64_t n) { return static_cast<size_t>((n + 3) / 4 * 4); }

size_t workspace_ints(int32_t rows, int64_t pages) {
    return ints(tiles_of(pages)) + 4 + ints(2 * (int64_t(rows) + 1)) + 3 * ints(rows) + 3 * ints(pages);
}

aq_status check_pages(int32_t n, int32_t num_rows, int32_t max_pages, int64_t num_pages) {
    if (n < 0 || num_rows < 0 || max_pages < 0 || num_pages < 0) return AQ_ERR_INVALID_ARGUMENT;
    if (num_pages > 0x7fff0000ll) return AQ_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_pages) * kPage > 0x7fffffffll) return AQ_ERR_UNSUPPORTED;
    return AQ_OK;
}

aq_status check_pools(const aq_page_pool *pools, int32_t num_pools) {
    if (num_pools < 0 || (num_pools > 0 && !pools)) return AQ_ERR_INVALID_ARGUMENT;
    if (num_pools > kMaxPools) return AQ_ERR_UNSUPPORTED;
    for (int k = 0; k < num_pools; ++k)
        if (!pools[k].data || off16(pools[k].data) || pools[k].page_bytes < 4 || pools[k].page_bytes % 4)
            return AQ_ERR_INVALID_ARGUMENT;
    for (int k = 0; k < num_pools; ++k)                // (chunks are counted in 32 bits)
        if (pools[k].page_bytes > (1ll << 34)) return AQ_ERR_UNSUPPORTED;
    return AQ_OK;
}

PageParams page_params(int32_t n, const int32_t *rows, const int32_t *args, int32_t *block_table, int32_t num_rows,
                       int32_t max_pages, int32_t *seq_lens, int32_t *refcount, int64_t num_pages, void *workspace,
                       int32_t *status) {
    PageParams p{};
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.refcount = refcount;
    p.rows = rows;
    p.args = args;
    p.status = status;
    p.n = n;
    p.num_rows = num_rows;
    p.max_pages = max_pages;
    p.num_pages = static_cast<int32_t>(num_pages);
    p.ntiles = tiles_of(num_pages);
    int32_t *w = static_cast<int32_t *>(workspace);
    if (w) {
        p.tiles = w;
        p.total = p.tiles + ints(p.ntiles);
        p.off = reinterpret_cast<long long *>(p.total + 4);
        p.info = p.total + 4 + ints(2 * (int64_t(num_rows) + 1));
        p.claim = p.info + ints(num_rows);
        p.from = p.claim + ints(num_rows);
        p.rank = p.from + ints(num_rows);
        p.movers = p.rank + ints(num_pages);
        p.holes = p.movers + ints(num_pages);
    }
    return p;
}

PagePools page_pools(const aq_page_pool *pools, int32_t num_pools) {
    PagePools pl{};
    pl.n = num_pools;
    for (int k = 0; k < num_pools; ++k) {
        pl.pool[k] = pools[k];
        pl.first[k + 1] = pl.first[k] + static_cast<int32_t>((pools[k].page_bytes + kChunk - 1) / kChunk);
    }
    return pl;
}

aq_status done(cudaError_t e) {
    if (e == cudaSuccess) return AQ_OK;
    record_cuda_error(e);
    return AQ_ERR_CUDA;
}

}  // namespace

}  // namespace aq

using namespace aq;

extern "C" {

aq_status aq_pages_workspace(int32_t num_rows, int64_t num_pages, size_t *workspace_bytes) {
    const aq_status st = check_pages(0, num_rows, 0, num_pages);
    if (st != AQ_OK) return st;
    if (!workspace_bytes) return AQ_ERR_INVALID_ARGUMENT;
    *workspace_bytes = workspace_ints(num_rows, num_pages) * sizeof(int32_t);
    return AQ_OK;
}

aq_status aq_pages_extend(int32_t n, const int32_t *rows, const int32_t *new_lens, int32_t *block_table,
                          int32_t num_rows, int32_t max_pages, int32_t *seq_lens, int32_t *refcount,
                          int64_t num_pages, const aq_page_pool *pools, int32_t num_pools, void *workspace,
                          size_t workspace_bytes, int32_t *device_status, aq_stream_t stream) {
    aq_status st = check_pages(n, num_rows, max_pages, num_pages);
    if (st == AQ_OK) st = check_pools(pools, num_pools);
    if (st != AQ_OK) return st;
    if (n == 0) return AQ_OK;
    if (n > num_rows || !rows || !new_lens || !block_table || !seq_lens || (num_pages > 0 && !refcount) || off16(refcount))
        return AQ_ERR_INVALID_ARGUMENT;
    if (!workspace || workspace_bytes < workspace_ints(num_rows, num_pages) * sizeof(int32_t))
        return AQ_ERR_WORKSPACE_TOO_SMALL;
    if (off16(workspace)) return AQ_ERR_INVALID_ARGUMENT;
    const PageParams p = page_params(n, rows, new_lens, block_table, num_rows, max_pages, seq_lens, refcount, num_pages,
                                     workspace, device_status);
    const PagePools pl = page_pools(pools, num_pools);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // a page's chunks over at most 64 CTAs of 8 warps
    const int parts = (pl.first[num_pools] + 7) / 8;
    cudaError_t e = cudaSuccess;
    if (p.ntiles > kDirectTiles) e = launch_dependent(pages_count_kernel<true>, dim3(p.ntiles), dim3(kThreads), 0, s, 1, p);
    if (e == cudaSuccess) e = launch_dependent(pages_assign_kernel, dim3(p.ntiles + 1), dim3(kThreads), 0, s, 1, p);
    if (e == cudaSuccess)
        e = launch_dependent(pages_grow_kernel, dim3(n, parts < 1 ? 1 : parts > 64 ? 64 : parts), dim3(kCopyThreads), 0, s,
                             1, p, pl);
    return done(e);
}

aq_status aq_pages_fork(int32_t n, const int32_t *src_rows, const int32_t *dst_rows, int32_t *block_table,
                        int32_t num_rows, int32_t max_pages, int32_t *seq_lens, int32_t *refcount,
                        int64_t num_pages, int32_t *device_status, aq_stream_t stream) {
    const aq_status st = check_pages(n, num_rows, max_pages, num_pages);
    if (st != AQ_OK) return st;
    if (n == 0) return AQ_OK;
    if (n > num_rows || !src_rows || !dst_rows || !block_table || !seq_lens || (num_pages > 0 && !refcount) || off16(refcount))
        return AQ_ERR_INVALID_ARGUMENT;
    const PageParams p = page_params(n, src_rows, dst_rows, block_table, num_rows, max_pages, seq_lens, refcount,
                                     num_pages, nullptr, device_status);
    return done(launch_dependent(pages_fork_kernel, dim3(n), dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream), 1, p));
}

aq_status aq_pages_free(int32_t n, const int32_t *rows, const int32_t *keep_lens, int32_t *block_table,
                        int32_t num_rows, int32_t max_pages, int32_t *seq_lens, int32_t *refcount,
                        int64_t num_pages, int32_t *device_status, aq_stream_t stream) {
    const aq_status st = check_pages(n, num_rows, max_pages, num_pages);
    if (st != AQ_OK) return st;
    if (n == 0) return AQ_OK;
    if (!rows || !block_table || !seq_lens || (num_pages > 0 && !refcount) || off16(refcount)) return AQ_ERR_INVALID_ARGUMENT;
    const PageParams p = page_params(n, rows, keep_lens, block_table, num_rows, max_pages, seq_lens, refcount,
                                     num_pages, nullptr, device_status);
    return done(launch_dependent(pages_free_kernel, dim3(n), dim3(kCopyThreads), 0, reinterpret_cast<cudaStream_t>(stream),
                                 1, p));
}

aq_status aq_pages_compact(int32_t *block_table, int32_t num_rows, int32_t max_pages, int32_t *seq_lens,
                           int32_t *refcount, int64_t num_pages, const aq_page_pool *pools, int32_t num_pools,
                           void *workspace, size_t workspace_bytes, int32_t *device_status, aq_stream_t stream) {
    aq_status st = check_pages(0, num_rows, max_pages, num_pages);
    if (st == AQ_OK) st = check_pools(pools, num_pools);
    if (st != AQ_OK) return st;
    if (num_pages == 0) return AQ_OK;
    if (!refcount || off16(refcount) || (num_rows > 0 && (!block_table || !seq_lens))) return AQ_ERR_INVALID_ARGUMENT;
    if (!workspace || workspace_bytes < workspace_ints(num_rows, num_pages) * sizeof(int32_t))
        return AQ_ERR_WORKSPACE_TOO_SMALL;
    if (off16(workspace)) return AQ_ERR_INVALID_ARGUMENT;
    const PageParams p = page_params(0, nullptr, nullptr, block_table, num_rows, max_pages, seq_lens, refcount, num_pages,
                                     workspace, device_status);
    const PagePools pl = page_pools(pools, num_pools);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int table = num_rows < 152 ? num_rows : 152;
    cudaError_t e = cudaSuccess;
    if (p.ntiles > kDirectTiles) e = launch_dependent(pages_count_kernel<false>, dim3(p.ntiles), dim3(kThreads), 0, s, 1, p);
    if (e == cudaSuccess) e = launch_dependent(pages_map_kernel, dim3(p.ntiles), dim3(kThreads), 0, s, 1, p);
    if (e == cudaSuccess)
        e = launch_dependent(pages_move_kernel, dim3(table + 152 * 5), dim3(kCopyThreads), 0, s, 1, p, pl, table);
    return done(e);
}

}  // extern "C"
