// Maintenance of a paged cache of FP16 keys and values: writing new tokens,
// and reserving, forking, freeing, compacting and copying pages.
//
// The bookkeeping (page tables, lengths, reference counts) lives in device
// memory and is changed by kernels, so that a serving loop never waits for the
// host.  Free pages are taken lowest number first in the order of the
// requests.  That needs the rank of each free page among the free ones, a
// prefix sum over the reference counts, which one CTA computes (4 bytes a
// page); everything that moves data or whole tables is spread over the GPU in
// a second launch.  Every page and row number read from memory is checked
// against its range before it is used as an address.
#include <cuda_fp16.h>

#include <mutex>

#include "internal.h"
#include "ptx.cuh"

namespace compfp32 {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanItems = 2;                             // entries a thread takes of a plan tile
constexpr int kPlanTile = kPlanThreads * kPlanItems;
constexpr int kRowThreads = 128;
constexpr int kCopyThreads = 256;

// Exclusive prefix sum of v over the CTA (kPlanThreads threads), and its total.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();  // warp_sums may still be read from the call before
    if (lane == 31)
        warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o)
                s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    total = warp_sums[31];
    return x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// The number of free pages; refs_out = refs on the way where they differ.
__device__ int64_t count_free(const int32_t* refs, int32_t* refs_out, int64_t pages, int* warp_sums)
{
    int n = 0;  // a thread sees at most pages / kPlanThreads of them
    for (int64_t p = threadIdx.x; p < pages; p += kPlanThreads) {
        const int32_t r = refs[p];
        n += r == 0;
        if (refs_out != refs)
            refs_out[p] = r;
    }
    int total;
    (void)block_scan(n, warp_sums, total);
    return total;
}

// Calls use(rank, page) for the `need` lowest free pages in ascending order.
template <typename Use>
__device__ void take_free(const int32_t* refs, int64_t pages, int64_t need, int* warp_sums, Use use)
{
    int64_t done = 0;
    for (int64_t p0 = 0; p0 < pages && done < need; p0 += kPlanTile) {
        const int64_t p = p0 + threadIdx.x * kPlanItems;
        bool free[kPlanItems];
        int n = 0, total;
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i) {
            free[i] = p + i < pages && refs[p + i] == 0;
            n += free[i];
        }
        int64_t rank = done + block_scan(n, warp_sums, total);
#pragma unroll
        for (int i = 0; i < kPlanItems; ++i)
            if (free[i]) {
                if (rank < need)
                    use(rank, p + i);
                ++rank;
            }
        done += total;
    }
}

// How a row is forked: its full pages, and the tokens in its partly filled one.
struct Fork {
    int parent, full, rest;  // parent < 0: not to be done
};

__device__ __forceinline__ Fork fork_of(int32_t parent, int32_t child, const int32_t* lengths, int64_t rows,
                                        int64_t width, int page_size)
{
    Fork f{-1, 0, 0};
    if (parent < 0 || parent >= rows || child < 0 || child >= rows)
        return f;
    int64_t n = lengths[parent];
    n = n < 0 ? 0 : (n > width * page_size ? width * page_size : n);
    f.parent = parent;
    f.full = static_cast<int>(n / page_size);
    f.rest = static_cast<int>(n % page_size);
    return f;
}

struct Tables {
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* refs;
    int32_t* table_out;
    int32_t* lengths_out;
    int32_t* refs_out;
    int64_t rows, width, pages;
    int page_size;
};

// First launch of a fork: which new page each child with a partly filled last
// page gets, or that there are not enough.  rank_child: n ints.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(Tables t, const int32_t* parents,
                                                                 const int32_t* children, int n, int32_t* left)
{
    extern __shared__ int rank_child[];
    __shared__ int warp_sums[32];
    int need = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + static_cast<int>(threadIdx.x);
        bool wants = false;
        if (i < n) {
            const Fork f = fork_of(parents[i], children[i], t.lengths, t.rows, t.width, t.page_size);
            wants = f.parent >= 0 && f.rest > 0;
        }
        int total;
        const int at = need + block_scan(wants, warp_sums, total);
        if (wants)
            rank_child[at] = i;
        need += total;
    }
    const int64_t spare = count_free(t.refs, t.refs_out, t.pages, warp_sums) - need;
    if (threadIdx.x == 0)
        left[0] = static_cast<int32_t>(spare);
    if (spare < 0)
        return;
    __syncthreads();  // rank_child, and refs_out's copy, are complete
    take_free(t.refs, t.pages, need, warp_sums, [&](int64_t rank, int64_t page) {
        const int i = rank_child[rank];
        const Fork f = fork_of(parents[i], children[i], t.lengths, t.rows, t.width, t.page_size);
        t.table_out[children[i] * t.width + f.full] = static_cast<int32_t>(page);
        t.refs_out[page] = 1;
    });
}

// The index i < n with list[i] == row, or -1 (the last one, if there are several).
__device__ __forceinline__ int find_row(const int32_t* list, int n, int64_t row, int* found)
{
    if (threadIdx.x == 0)
        *found = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if (list[i] == row)
            atomicMax(found, i);
    __syncthreads();
    return *found;
}

// 16-byte copies: element i of the CTA's share, `ctas` CTAs together.
__device__ __forceinline__ void copy16(const uint4* src, uint4* dst, int64_t n, int cta, int ctas)
{
    const int64_t step = static_cast<int64_t>(ctas) * blockDim.x;
    int64_t i = static_cast<int64_t>(cta) * blockDim.x + threadIdx.x;
    for (; i + 3 * step < n; i += 4 * step) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = __ldcs(src + i + j * step);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            dst[i + j * step] = v[j];
    }
    for (; i < n; i += step)
        dst[i] = __ldcs(src + i);
}

// Second launch: one CTA for each row (tables, lengths, counts of the shared
// pages), then `ctas` for each child (the filled tokens of its last page).
__global__ void __launch_bounds__(kCopyThreads) fork_copy_kernel(Tables t, comp_kv_cache_t cache,
                                                                 const int32_t* parents, const int32_t* children,
                                                                 int n, int ctas, const int32_t* left)
{
    __shared__ int found;
    const bool enough = left[0] >= 0;
    if (blockIdx.x < t.rows) {
        const int64_t row = blockIdx.x;
        const int i = find_row(children, n, row, &found);
        const Fork f = i < 0 ? Fork{-1, 0, 0}
                             : fork_of(parents[i], children[i], t.lengths, t.rows, t.width, t.page_size);
        const int64_t at = row * t.width;
        if (f.parent < 0 || !enough) {
            if (t.table_out != t.table)
                for (int64_t c = threadIdx.x; c < t.width; c += blockDim.x)
                    t.table_out[at + c] = t.table[at + c];
            if (threadIdx.x == 0 && t.lengths_out != t.lengths)
                t.lengths_out[row] = t.lengths[row];
            return;
        }
        const int32_t* const from = t.table + f.parent * t.width;
        for (int64_t c = threadIdx.x; c < t.width; c += blockDim.x) {
            if (c == f.full && f.rest > 0)
                continue;  // the new page
            const int32_t page = c < f.full ? from[c] : -1;
            t.table_out[at + c] = page;
            if (page >= 0 && page < t.pages)
                atomicAdd(t.refs_out + page, 1);
        }
        if (threadIdx.x == 0)
            t.lengths_out[row] = f.full * t.page_size + f.rest;
        return;
    }
    const int i = static_cast<int>((blockIdx.x - t.rows) / ctas);
    const int cta = static_cast<int>((blockIdx.x - t.rows) % ctas);
    const Fork f = fork_of(parents[i], children[i], t.lengths, t.rows, t.width, t.page_size);
    if (!enough || f.parent < 0 || f.rest == 0)
        return;
    const int32_t src = t.table[f.parent * t.width + f.full], dst = t.table_out[children[i] * t.width + f.full];
    if (dst < 0 || dst >= t.pages)
        return;
    const bool there = src >= 0 && src < t.pages;  // if not it reads as zeros, and so must its copy
    const int64_t head = static_cast<int64_t>(t.page_size) * cache.head_dim / 8;  // uint4s
    for (int u = cta; u < 2 * cache.kv_heads; u += ctas) {
        uint4* const base = reinterpret_cast<uint4*>(u < cache.kv_heads ? cache.k : cache.v);
        const int64_t h = u < cache.kv_heads ? u : u - cache.kv_heads;
        uint4* const to = base + (dst * static_cast<int64_t>(cache.kv_heads) + h) * head;
        const int64_t n = static_cast<int64_t>(f.rest) * cache.head_dim / 8;
        if (there)
            copy16(base + (src * static_cast<int64_t>(cache.kv_heads) + h) * head, to, n, 0, 1);
        else
            for (int64_t i = threadIdx.x; i < n; i += blockDim.x)
                to[i] = make_uint4(0, 0, 0, 0);
    }
}

__global__ void __launch_bounds__(kCopyThreads) copy_ints_kernel(const int32_t* src, int32_t* dst, int64_t n)
{
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        dst[i] = src[i];
}

// One CTA for each row.
__global__ void __launch_bounds__(kRowThreads) free_kernel(Tables t, const int32_t* seqs, int n)
{
    __shared__ int found;
    const int64_t row = blockIdx.x, at = row * t.width;
    const bool gone = find_row(seqs, n, row, &found) >= 0;
    for (int64_t c = threadIdx.x; c < t.width; c += blockDim.x) {
        const int32_t page = t.table[at + c];
        if (gone && page >= 0 && page < t.pages && atomicSub(t.refs_out + page, 1) <= 0)
            atomicAdd(t.refs_out + page, 1);  // it was free already: stays at 0
        if (gone || t.table_out != t.table)
            t.table_out[at + c] = gone ? -1 : page;
    }
    if (threadIdx.x == 0 && (gone || t.lengths_out != t.lengths))
        t.lengths_out[row] = gone ? 0 : t.lengths[row];
}

// The same for small tables by one CTA, in one launch: the counts first, then
// the rows.
__global__ void __launch_bounds__(kPlanThreads) free_small_kernel(Tables t, const int32_t* seqs, int n)
{
    if (t.refs_out != t.refs)
        for (int64_t p = threadIdx.x; p < t.pages; p += kPlanThreads)
            t.refs_out[p] = t.refs[p];
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for (int64_t row = threadIdx.x >> 5; row < t.rows; row += kPlanThreads / 32) {
        bool mine = false;
        for (int i = lane; i < n; i += 32)
            mine |= seqs[i] == row;
        const bool gone = __any_sync(0xffffffffu, mine);
        for (int64_t c = lane; c < t.width; c += 32) {
            const int32_t page = t.table[row * t.width + c];
            if (gone && page >= 0 && page < t.pages && atomicSub(t.refs_out + page, 1) <= 0)
                atomicAdd(t.refs_out + page, 1);
            if (gone || t.table_out != t.table)
                t.table_out[row * t.width + c] = gone ? -1 : page;
        }
        if (lane == 0 && (gone || t.lengths_out != t.lengths))
            t.lengths_out[row] = gone ? 0 : t.lengths[row];
    }
}

// Pages a row has (its leading entries that are not -1) and lacks for `want` tokens.
__device__ __forceinline__ void row_pages(const Tables& t, int64_t row, int32_t want, int& have, int& lack)
{
    int64_t lo = 0, hi = t.width;
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (t.table[row * t.width + mid] >= 0)
            lo = mid + 1;
        else
            hi = mid;
    }
    int64_t target = want <= 0 ? 0 : (static_cast<int64_t>(want) + t.page_size - 1) / t.page_size;
    target = target > t.width ? t.width : target;
    have = static_cast<int>(lo);
    lack = target > lo ? static_cast<int>(target - lo) : 0;
}

// One CTA.  t.lengths holds the wanted lengths; table_out and refs_out hold
// copies of (or are) table and refs; rows * width is an int.  Shared memory:
// 2 * rows ints.
__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(Tables t, int32_t* left)
{
    extern __shared__ int base[];  // first rank of each row's new pages
    int* const have = base + t.rows;
    __shared__ int warp_sums[32];
    int64_t need = 0;
    for (int64_t r0 = 0; r0 < t.rows; r0 += kPlanThreads) {
        const int64_t r = r0 + threadIdx.x;
        int mine = 0, lack = 0, total;
        if (r < t.rows)
            row_pages(t, r, t.lengths[r], mine, lack);
        const int at = block_scan(lack, warp_sums, total);
        if (r < t.rows) {
            base[r] = static_cast<int>(need) + at;
            have[r] = mine;
        }
        need += total;
    }
    const int64_t spare = count_free(t.refs, t.refs_out, t.pages, warp_sums) - need;
    if (threadIdx.x == 0)
        left[0] = spare < INT32_MIN ? INT32_MIN : static_cast<int32_t>(spare);
    if (spare < 0)
        return;
    __syncthreads();
    take_free(t.refs, t.pages, need, warp_sums, [&](int64_t rank, int64_t page) {
        // The last row whose first rank is not beyond this one: rows that take
        // nothing share the first rank of the row after them.
        int lo = 0, hi = static_cast<int>(t.rows) - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (base[mid] <= rank)
                lo = mid;
            else
                hi = mid - 1;
        }
        t.table_out[lo * t.width + have[lo] + (rank - base[lo])] = static_cast<int32_t>(page);
        t.refs_out[page] = 1;
    });
}

// First launch of a compaction, one CTA: remap and the count.  The j-th page
// in use at or beyond `live` goes to the j-th free page below it; there are
// equally many of both.  Two queues, one filled from each end of the pool,
// are paired as they fill.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const int32_t* refs, int64_t pages,
                                                                    int32_t* remap, int32_t* live_out)
{
    __shared__ int warp_sums[32];
    __shared__ int32_t holes[2 * kPlanTile], movers[2 * kPlanTile];
    int n = 0, live;
    for (int64_t p = threadIdx.x; p < pages; p += kPlanThreads)
        n += refs[p] > 0;
    (void)block_scan(n, warp_sums, live);
    if (threadIdx.x == 0)
        live_out[0] = live;
    int64_t ph = 0, pm = live;
    int nh = 0, nm = 0;
    while (ph < live || pm < pages || (nh > 0 && nm > 0)) {
        const int64_t before = ph + pm;
        // one tile from each end into its queue, where there is room
        for (int side = 0; side < 2; ++side) {
            int64_t& p0 = side ? pm : ph;
            const int64_t end = side ? pages : live;
            int& count = side ? nm : nh;
            if (p0 >= end || count > kPlanTile)
                continue;
            const int64_t p = p0 + threadIdx.x * kPlanItems;
            bool take[kPlanItems];
            int mine = 0, total;
#pragma unroll
            for (int i = 0; i < kPlanItems; ++i) {
                const bool in = p + i < end;
                const bool used = in && refs[p + i] > 0;
                take[i] = in && (side ? used : !used);
                mine += take[i];
                if (in && !(side && used))  // movers get theirs below
                    remap[p + i] = used ? static_cast<int32_t>(p + i) : -1;
            }
            int at = count + block_scan(mine, warp_sums, total);
#pragma unroll
            for (int i = 0; i < kPlanItems; ++i)
                if (take[i])
                    (side ? movers : holes)[at++] = static_cast<int32_t>(p + i);
            count += total;
            p0 += kPlanTile;
        }
        __syncthreads();
        const int m = nh < nm ? nh : nm;
        if (m == 0 && ph + pm == before)
            break;  // only if refs changed meanwhile: both ends have equally many
        for (int i = threadIdx.x; i < m; i += kPlanThreads)
            remap[movers[i]] = holes[i];
        // what is left moves to the front (at most 2 * kPlanTile entries)
        int32_t rest[2 * kPlanItems];
        int32_t* const queue = nh > nm ? holes : movers;
        const int keep = (nh > nm ? nh : nm) - m;
#pragma unroll
        for (int j = 0; j < 2 * kPlanItems; ++j) {
            const int i = static_cast<int>(threadIdx.x) + j * kPlanThreads;
            rest[j] = i < keep ? queue[m + i] : 0;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2 * kPlanItems; ++j) {
            const int i = static_cast<int>(threadIdx.x) + j * kPlanThreads;
            if (i < keep)
                queue[i] = rest[j];
        }
        __syncthreads();
        nh -= m;
        nm -= m;
    }
}

// Copies of `n` pages, spread over the grid in pieces of kPiece uint4s:
// page_of(i, src, dst) says whether the i-th is to be done.
constexpr int64_t kPiece = 4 * kCopyThreads;

template <typename PageOf>
__device__ __forceinline__ void copy_pages(const comp_kv_cache_t& cache, int64_t n, PageOf page_of)
{
    const int64_t vecs = static_cast<int64_t>(cache.kv_heads) * cache.page_size * cache.head_dim / 8;
    const int64_t pieces = (vecs + kPiece - 1) / kPiece;
    for (int64_t u = blockIdx.x; u < n * 2 * pieces; u += gridDim.x) {
        const int64_t i = u / (2 * pieces);
        const int64_t piece = u % (2 * pieces);
        int64_t src, dst;
        if (!page_of(i, src, dst))
            continue;
        uint4* const base = reinterpret_cast<uint4*>(piece < pieces ? cache.k : cache.v);
        const int64_t first = (piece % pieces) * kPiece;
        copy16(base + src * vecs + first, base + dst * vecs + first, vecs - first < kPiece ? vecs - first : kPiece, 0,
               1);
    }
}

// Second launch: the pages that move, the table and the counts renumbered.
__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(Tables t, comp_kv_cache_t cache,
                                                                    const int32_t* remap, const int32_t* live_in)
{
    const int64_t live = live_in[0];
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    for (int64_t i = first; i < t.rows * t.width; i += step) {
        const int32_t p = t.table[i];
        t.table_out[i] = p >= 0 && p < t.pages ? remap[p] : -1;
    }
    for (int64_t p = first; p < t.pages; p += step) {
        const int32_t r = t.refs[p], to = remap[p];
        if (p >= live) {
            if (to >= 0)
                t.refs_out[to] = r;
            t.refs_out[p] = 0;
        } else if (to >= 0) {
            t.refs_out[p] = r;
        }
    }
    copy_pages(cache, t.pages - live, [&](int64_t i, int64_t& src, int64_t& dst) {
        src = live + i;
        dst = remap[src];
        return dst >= 0;
    });
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(comp_kv_cache_t cache, const int32_t* from,
                                                                  const int32_t* to, int64_t n)
{
    copy_pages(cache, n, [&](int64_t i, int64_t& src, int64_t& dst) {
        src = from[i];
        dst = to[i];
        return src >= 0 && src < cache.pages && dst >= 0 && dst < cache.pages;
    });
}

// New tokens into the cache: a thread rounds eight values of one token's head.
__global__ void __launch_bounds__(kCopyThreads) append_kernel(comp_kv_cache_t cache, const float* k, const float* v,
                                                              int64_t k_token, int64_t k_head, int64_t v_token,
                                                              int64_t v_head, int64_t total, const int32_t* table,
                                                              int64_t rows, int64_t width, const int32_t* cu,
                                                              const int32_t* start)
{
    grid_dependency_launch();
    const int parts = cache.head_dim / 8;
    const int64_t work = total * cache.kv_heads * parts;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; u < work;
         u += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int part = static_cast<int>(u % parts);
        const int64_t head = u / parts % cache.kv_heads, token = u / parts / cache.kv_heads;
        int64_t row = token, at = 0;
        if (cu) {  // the last row that begins at or before this token
            int64_t lo = 0, hi = rows - 1;
            while (lo < hi) {
                const int64_t mid = (lo + hi + 1) / 2;
                if (cu[mid] <= token)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            row = lo;
            at = token - cu[lo];
            if (at < 0 || token >= cu[lo + 1])
                continue;
        }
        at += start[row];
        const int64_t col = at / cache.page_size;
        if (at < 0 || col >= width)
            continue;
        const int32_t page = table[row * width + col];
        if (page < 0 || page >= cache.pages)
            continue;
        const int64_t to = ((page * static_cast<int64_t>(cache.kv_heads) + head) * cache.page_size +
                            at % cache.page_size) * cache.head_dim + part * 8;
        const float* const kp = k + token * k_token + head * k_head + part * 8;
        const float* const vp = v + token * v_token + head * v_head + part * 8;
        __half2 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = __floats2half2_rn(kp[2 * i], kp[2 * i + 1]);
            b[i] = __floats2half2_rn(vp[2 * i], vp[2 * i + 1]);
        }
        *reinterpret_cast<uint4*>(cache.k + to) = *reinterpret_cast<uint4*>(a);
        *reinterpret_cast<uint4*>(cache.v + to) = *reinterpret_cast<uint4*>(b);
    }
}

// One array of a call: `out` ones may share memory with nothing but the input
// that they may be (`same`).
struct Range {
    const void* p;
    int64_t bytes;
    const void* same = nullptr;
    bool out = false;
};

template <int N>
bool ranges_ok(const Range (&r)[N])
{
    for (int i = 0; i < N; ++i)
        if (r[i].bytes > 0 && !r[i].p)
            return false;
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j)
            if (i != j && r[i].out && !(r[i].p == r[i].same && r[j].p == r[i].same) &&
                overlap(r[i].p, r[i].bytes, r[j].p, r[j].bytes))
                return false;
    return true;
}

constexpr int64_t kMostListed = 32768;   // children of one fork (their ranks are kept in shared memory)
constexpr int64_t kMostRows = 16384;     // rows of one reserve (likewise)
constexpr int64_t kMostPages = INT32_MAX / 2;
// Counts, entries and comparisons that one CTA goes through sooner than a
// second launch begins (3.5 us for 6800 of them on the device, as two launches
// take, and 1.6 us less of host time; 4.5 us for 13000).
constexpr int64_t kSmallFree = 8192;

unsigned grid_of(int64_t work, int64_t per, const DeviceInfo& dev, int per_sm)
{
    const int64_t most = static_cast<int64_t>(dev.sm_count) * per_sm, g = (work + per - 1) / per;
    return static_cast<unsigned>(g < 1 ? 1 : (g > most ? most : g));
}

// A plan kernel's shared memory, raised once per device to the most that it may be
// asked for: another call may be about to launch with more than this one needs.
template <typename Kernel>
bool allow_smem(Kernel kernel, int64_t most, std::mutex& mu, bool (&done)[64], const DeviceInfo& dev)
{
    std::lock_guard<std::mutex> lock(mu);
    if (dev.device < 0 || dev.device >= 64)
        return false;
    if (!done[dev.device]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most)) !=
            cudaSuccess) {
            (void)cudaGetLastError();
            return false;
        }
        done[dev.device] = true;
    }
    return true;
}

comp_status_t copy_ints(const int32_t* src, int32_t* dst, int64_t n, const DeviceInfo& dev, cudaStream_t s)
{
    if (n == 0 || src == dst)
        return COMP_OK;
    copy_ints_kernel<<<grid_of(n, kCopyThreads, dev, 8), kCopyThreads, 0, s>>>(src, dst, n);
    return launch_status();
}

bool table_ok(int64_t pages, int page_size, int64_t rows, int64_t width, int64_t* entries)
{
    return pages >= 0 && pages <= kMostPages && (page_size == 16 || page_size == 32 || page_size == 64 ||
           page_size == 128) && rows >= 0 && rows <= INT32_MAX / 2 && width >= 0 &&
           width <= INT32_MAX / (2 * page_size) && mul_ok(rows, width, entries) && *entries <= INT64_MAX / 8;
}

}  // namespace

bool kv_cache_ok(const comp_kv_cache_t* c, int64_t* bytes)
{
    if (!c || c->pages < 0 || c->pages > kMostPages || c->kv_heads <= 0 || c->kv_heads > 65535 || c->head_dim <= 0 ||
        c->head_dim > 128 || c->head_dim % 8 != 0)
        return false;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return false;
    const int64_t page = static_cast<int64_t>(c->kv_heads) * c->page_size * c->head_dim * 2;
    if (!mul_ok(c->pages, page, bytes) || *bytes > INT64_MAX / 4)
        return false;
    if (*bytes > 0 && (!c->k || !c->v || (reinterpret_cast<uintptr_t>(c->k) & 15u) != 0 ||
                       (reinterpret_cast<uintptr_t>(c->v) & 15u) != 0 || overlap(c->k, *bytes, c->v, *bytes)))
        return false;
    return true;
}

}  // namespace compfp32

using namespace compfp32;

extern "C" {

comp_status_t comp_kv_append_f32(const comp_kv_cache_t* cache, const float* k, const float* v, int64_t k_token,
                                 int64_t k_head, int64_t v_token, int64_t v_head, int64_t total,
                                 const int32_t* table, int64_t rows, int64_t width, const int32_t* cu,
                                 const int32_t* start, comp_stream_t stream)
{
    int64_t bytes, entries;
    if (!kv_cache_ok(cache, &bytes) || !table_ok(cache->pages, cache->page_size, rows, width, &entries) ||
        total < 0 || total > INT32_MAX || (!cu && total != rows))
        return COMP_ERR_INVALID_VALUE;
    int64_t kb, vb;
    if (!strided_bytes(total, cache->kv_heads, cache->head_dim, k_token, k_head, 4, &kb) ||
        !strided_bytes(total, cache->kv_heads, cache->head_dim, v_token, v_head, 4, &vb))
        return COMP_ERR_INVALID_VALUE;
    if (total == 0 || bytes == 0 || entries == 0)
        return COMP_OK;
    const Range r[] = {{cache->k, bytes, nullptr, true}, {cache->v, bytes, nullptr, true}, {k, kb}, {v, vb},
                       {table, 4 * entries}, {cu, cu ? 4 * (rows + 1) : 0}, {start, 4 * rows}};
    if (!ranges_ok(r))
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    const comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    const int64_t work = total * cache->kv_heads * (cache->head_dim / 8);
    append_kernel<<<grid_of(work, kCopyThreads, dev, 8), kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        *cache, k, v, k_token, k_head, v_token, v_head, total, table, rows, width, cu, start);
    return launch_status();
}

comp_status_t comp_kv_reserve(int64_t pages, int32_t page_size, const int32_t* table, const int32_t* refs,
                              int64_t rows, int64_t width, const int32_t* want, int32_t* table_out,
                              int32_t* refs_out, int32_t* left, comp_stream_t stream)
{
    int64_t entries;
    if (!table_ok(pages, page_size, rows, width, &entries) || rows > kMostRows || entries > INT32_MAX)
        return COMP_ERR_INVALID_VALUE;
    const Range r[] = {{table, 4 * entries}, {refs, 4 * pages}, {want, 4 * rows},
                       {table_out, 4 * entries, table, true}, {refs_out, 4 * pages, refs, true},
                       {left, 4, nullptr, true}};
    if (!ranges_ok(r))
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = copy_ints(table, table_out, entries, dev, s);
    if (st != COMP_OK)
        return st;
    const size_t smem = static_cast<size_t>(8 * rows);
    static std::mutex mu;
    static bool done[64] = {};
    if (!allow_smem(reserve_kernel, 8 * kMostRows, mu, done, dev))
        return COMP_ERR_CUDA;
    reserve_kernel<<<1, kPlanThreads, smem, s>>>(
        Tables{table, want, refs, table_out, nullptr, refs_out, rows, width, pages, page_size}, left);
    return launch_status();
}

comp_status_t comp_kv_fork(const comp_kv_cache_t* cache, const int32_t* table, const int32_t* lengths,
                           const int32_t* refs, int64_t rows, int64_t width, const int32_t* parents,
                           const int32_t* children, int64_t n, int32_t* table_out, int32_t* lengths_out,
                           int32_t* refs_out, int32_t* left, comp_stream_t stream)
{
    int64_t bytes, entries;
    if (!kv_cache_ok(cache, &bytes) || !table_ok(cache->pages, cache->page_size, rows, width, &entries) || n < 0 ||
        n > kMostListed)
        return COMP_ERR_INVALID_VALUE;
    const int64_t pages = cache->pages;
    const Range r[] = {{cache->k, bytes, nullptr, true}, {cache->v, bytes, nullptr, true},
                       {table, 4 * entries}, {lengths, 4 * rows}, {refs, 4 * pages}, {parents, 4 * n},
                       {children, 4 * n}, {table_out, 4 * entries, table, true},
                       {lengths_out, 4 * rows, lengths, true}, {refs_out, 4 * pages, refs, true},
                       {left, 4, nullptr, true}};
    if (!ranges_ok(r))
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Tables t{table, lengths, refs, table_out, lengths_out, refs_out, rows, width, pages, cache->page_size};
    const size_t smem = static_cast<size_t>(4 * n);
    static std::mutex mu;
    static bool done[64] = {};
    if (!allow_smem(fork_plan_kernel, 4 * kMostListed, mu, done, dev))
        return COMP_ERR_CUDA;
    fork_plan_kernel<<<1, kPlanThreads, smem, s>>>(t, parents, children, static_cast<int>(n), left);
    st = launch_status();
    if (st != COMP_OK || rows == 0)
        return st;
    const int ctas = 2 * cache->kv_heads < 16 ? 2 * cache->kv_heads : 16;
    fork_copy_kernel<<<static_cast<unsigned>(rows + n * ctas), kCopyThreads, 0, s>>>(
        t, *cache, parents, children, static_cast<int>(n), ctas, left);
    return launch_status();
}

comp_status_t comp_kv_free(int64_t pages, const int32_t* table, const int32_t* lengths, const int32_t* refs,
                           int64_t rows, int64_t width, const int32_t* seqs, int64_t n, int32_t* table_out,
                           int32_t* lengths_out, int32_t* refs_out, comp_stream_t stream)
{
    int64_t entries;
    if (!table_ok(pages, 16, rows, width, &entries) || n < 0 || n > INT32_MAX / 2)
        return COMP_ERR_INVALID_VALUE;
    const Range r[] = {{table, 4 * entries}, {lengths, 4 * rows}, {refs, 4 * pages}, {seqs, 4 * n},
                       {table_out, 4 * entries, table, true}, {lengths_out, 4 * rows, lengths, true},
                       {refs_out, 4 * pages, refs, true}};
    if (!ranges_ok(r))
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Tables t{table, lengths, refs, table_out, lengths_out, refs_out, rows, width, pages, 16};
    if (pages + entries + rows * n <= kSmallFree) {
        free_small_kernel<<<1, kPlanThreads, 0, s>>>(t, seqs, static_cast<int>(n));
        return launch_status();
    }
    st = copy_ints(refs, refs_out, pages, dev, s);
    if (st != COMP_OK || rows == 0)
        return st;
    free_kernel<<<static_cast<unsigned>(rows), kRowThreads, 0, s>>>(t, seqs, static_cast<int>(n));
    return launch_status();
}

comp_status_t comp_kv_compact(const comp_kv_cache_t* cache, const int32_t* table, const int32_t* refs, int64_t rows,
                              int64_t width, int32_t* table_out, int32_t* refs_out, int32_t* remap, int32_t* live,
                              comp_stream_t stream)
{
    int64_t bytes, entries;
    if (!kv_cache_ok(cache, &bytes) || !table_ok(cache->pages, cache->page_size, rows, width, &entries))
        return COMP_ERR_INVALID_VALUE;
    const int64_t pages = cache->pages;
    const Range r[] = {{cache->k, bytes, nullptr, true}, {cache->v, bytes, nullptr, true}, {table, 4 * entries},
                       {refs, 4 * pages}, {table_out, 4 * entries, table, true}, {refs_out, 4 * pages, refs, true},
                       {remap, 4 * pages, nullptr, true}, {live, 4, nullptr, true}};
    if (!ranges_ok(r))
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    compact_plan_kernel<<<1, kPlanThreads, 0, s>>>(refs, pages, remap, live);
    st = launch_status();
    if (st != COMP_OK)
        return st;
    const Tables t{table, nullptr, refs, table_out, nullptr, refs_out, rows, width, pages, cache->page_size};
    compact_move_kernel<<<static_cast<unsigned>(dev.sm_count * 8), kCopyThreads, 0, s>>>(t, *cache, remap, live);
    return launch_status();
}

comp_status_t comp_kv_copy_pages(const comp_kv_cache_t* cache, const int32_t* src, const int32_t* dst, int64_t n,
                                 comp_stream_t stream)
{
    int64_t bytes;
    if (!kv_cache_ok(cache, &bytes) || n < 0 || n > kMostPages)
        return COMP_ERR_INVALID_VALUE;
    const Range r[] = {{cache->k, bytes, nullptr, true}, {cache->v, bytes, nullptr, true}, {src, 4 * n}, {dst, 4 * n}};
    if (!ranges_ok(r))
        return COMP_ERR_INVALID_VALUE;
    if (n == 0 || bytes == 0)
        return COMP_OK;
    DeviceInfo dev;
    const comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    const int64_t vecs = static_cast<int64_t>(cache->kv_heads) * cache->page_size * cache->head_dim / 8;
    const int64_t units = n * 2 * ((vecs + kPiece - 1) / kPiece);
    copy_pages_kernel<<<grid_of(units, 1, dev, 8), kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(*cache, src,
                                                                                                         dst, n);
    return launch_status();
}

}  // extern "C"
