// cache_pages.cu -- the pages of the cache: forking sequences, appending
// tokens, copying, collecting (freeing) and compacting pages.
//
// These operators compute nothing: they move rows of K and V and rewrite the
// tables that name them, so each is bound by the bytes it moves (HBM) or,
// when that is little, by its launches.  All bookkeeping runs on the device
// and depends only on the device's tables, so a serving loop (beam search,
// sampling from one prompt) can record the calls in a CUDA graph and never
// read a length back.  Three choices make every call repeatable and its
// result independent of the order in which blocks run:
//   * Tables and counters that change have separate inputs and outputs.  No
//     block reads what another block of the same launch writes, so each
//     block may work out the same allocation for itself (a scan over the
//     sequences, a microsecond) and one launch is enough.
//   * Pages are handed out by rank: the r-th page a call needs, in sequence
//     order, is free_pages[free_count - 1 - r].  No atomic decides who gets
//     which page.
//   * There are no reference counts to keep in step.  A page is in use if a
//     table entry below some sequence's length names it; fa_cache_collect
//     finds the others.  Sharing a page is naming it twice.
#include <climits>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {

namespace cache_impl {

constexpr int kPage = 16;          // tokens per page
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Both caches as rows of 16-byte words, and the FP8 scales beside them.
struct Pages {
    uint4 *k, *v;
    float *ks, *vs;        // [num_pages][Hkv] or nullptr
    int num_pages, Hkv;
    int tok16;             // 16-byte words per token (K or V)
};

__device__ __forceinline__ bool exists(const Pages &pg, int page) {
    return page >= 0 && page < pg.num_pages;
}
__device__ __forceinline__ int pages_of(int len) { return (len + kPage - 1) / kPage; }

// Sum of one value per thread; every thread gets the block's total.
__device__ __forceinline__ int block_sum(int x, int *s_warp) {
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();                       // s_warp may still be read from the call before
    if (lane_id() == 0) s_warp[warp_id()] = x;
    __syncthreads();
    int t = 0;
    #pragma unroll
    for (int w = 0; w < kWarps; ++w) t += s_warp[w];
    return t;
}

// Exclusive prefix sum over the block's threads; `total` gets the sum.
__device__ __forceinline__ int block_scan(int x, int *s_warp, int &total) {
    const int lane = lane_id(), warp = warp_id();
    int inc = x;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int before = 0;
    total = 0;
    #pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    return before + inc - x;
}

// n 16-byte words from src to dst (disjoint), four loads in flight per thread.
__device__ __forceinline__ void copy_words(uint4 *__restrict__ dst, const uint4 *__restrict__ src,
                                           int n) {
    int i = threadIdx.x;
    for (; i + 3 * kThreads < n; i += 4 * kThreads) {
        const uint4 a = __ldcs(src + i), b = __ldcs(src + i + kThreads);
        const uint4 c = __ldcs(src + i + 2 * kThreads), d = __ldcs(src + i + 3 * kThreads);
        __stcs(dst + i, a);
        __stcs(dst + i + kThreads, b);
        __stcs(dst + i + 2 * kThreads, c);
        __stcs(dst + i + 3 * kThreads, d);
    }
    for (; i < n; i += kThreads) __stcs(dst + i, __ldcs(src + i));
}

// The first `toks` tokens of page src to page dst, and src's scales.
__device__ __forceinline__ void copy_page(const Pages &pg, int src, int dst, int toks, bool do_k,
                                          bool do_v) {
    const size_t page16 = (size_t)kPage * pg.tok16;
    if (do_k) copy_words(pg.k + dst * page16, pg.k + src * page16, toks * pg.tok16);
    if (do_v) copy_words(pg.v + dst * page16, pg.v + src * page16, toks * pg.tok16);
    if (pg.ks) {
        for (int h = threadIdx.x; h < pg.Hkv; h += kThreads) {
            if (do_k) pg.ks[(size_t)dst * pg.Hkv + h] = pg.ks[(size_t)src * pg.Hkv + h];
            if (do_v) pg.vs[(size_t)dst * pg.Hkv + h] = pg.vs[(size_t)src * pg.Hkv + h];
        }
    }
}

// A length a table of max_pages can hold; others are reported and read as 0.
__device__ __forceinline__ int good_len(int len, int max_pages) {
    if (len < 0 || len > max_pages * kPage) {
        report_error(kDevErrInput);
        return 0;
    }
    return len;
}

__device__ __forceinline__ int good_count(const int *count, int capacity) {
    const int c = __ldg(count);
    if (c < 0 || c > capacity) {
        report_error(kDevErrInput);
        return 0;
    }
    return c;
}

// ------------------------------------------------------------------- fork
// Slot i of the new batch continues slot parents[i] of the old one.  Full
// pages are shared (their table entries copied); a partly filled last page
// stays with the first slot i that continues it, and every later one gets a
// fresh page with its tokens copied.  blockIdx.y = 0 copies K and writes the
// tables, 1 copies V.  Each block finds the first slot of every parent
// (shared-memory minimum) and counts the fresh pages before its own slots.
__global__ void __launch_bounds__(kThreads)
fork_kernel(Pages pg, const int *__restrict__ table, const int *__restrict__ lens,
            const int *__restrict__ parents, const int *__restrict__ free_pages,
            const int *__restrict__ free_count, int free_capacity, int *__restrict__ table_out,
            int *__restrict__ lens_out, int *__restrict__ count_out, int slots_in, int slots_out,
            int max_pages, int per_block) {
    extern __shared__ int s_first[];
    __shared__ int s_warp[kWarps];
    const int tid = threadIdx.x;
    for (int s = tid; s < slots_in; s += kThreads) s_first[s] = INT_MAX;
    __syncthreads();
    for (int i = tid; i < slots_out; i += kThreads) {
        const int p = __ldg(parents + i);
        if (p >= 0 && p < slots_in)
            atomicMin(&s_first[p], i);
        else if (p != -1)
            report_error(kDevErrInput);
    }
    __syncthreads();
    auto copies = [&](int i) -> int {      // 1 if slot i needs a fresh page
        const int p = __ldg(parents + i);
        if (p < 0 || p >= slots_in) return 0;
        const int len = good_len(__ldg(lens + p), max_pages);
        return (len % kPage != 0 && s_first[p] != i) ? 1 : 0;
    };
    const int e0 = blockIdx.x * per_block, e1 = min(slots_out, e0 + per_block);
    int before = 0, all = 0;
    for (int i = tid; i < slots_out; i += kThreads) {
        const int c = copies(i);
        all += c;
        if (i < e0) before += c;
    }
    int rank = block_sum(before, s_warp);
    const int count = good_count(free_count, free_capacity);
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        all = block_sum(all, s_warp);
        if (tid == 0) *count_out = count - min(all, count);
    }
    for (int i = e0; i < e1; ++i) {        // uniform over the block
        const int p = __ldg(parents + i);
        int len = (p >= 0 && p < slots_in) ? good_len(__ldg(lens + p), max_pages) : 0;
        const int rest = len % kPage;
        int fresh = -1;
        if (copies(i)) {
            const int r = rank++;
            if (r < count) fresh = __ldg(free_pages + count - 1 - r);
            if (r >= count || !exists(pg, fresh)) {
                report_error(r >= count ? kDevErrPages : kDevErrInput);
                fresh = -1;
                len = 0;                   // the slot stays empty
            }
        }
        const int used = pages_of(len);
        const int *row = table + (size_t)(p < 0 ? 0 : p) * max_pages;
        if (blockIdx.y == 0) {
            // (so does one whose parent names a page that does not exist)
            bool bad = false;
            for (int c = tid; c < used; c += kThreads) bad |= !exists(pg, __ldg(row + c));
            const bool keep = !__syncthreads_or(bad);
            for (int c = tid; keep && c < used; c += kThreads)
                table_out[(size_t)i * max_pages + c] = (fresh >= 0 && c == used - 1) ? fresh : __ldg(row + c);
            if (tid == 0) {
                lens_out[i] = keep ? len : 0;
                if (!keep) report_error(kDevErrInput);
            }
        }
        if (fresh >= 0) {
            const int src = __ldg(row + used - 1);
            if (exists(pg, src) && src != fresh)
                copy_page(pg, src, fresh, rest, blockIdx.y == 0, blockIdx.y == 1);
        }
    }
}

// ----------------------------------------------------------------- append
// Writes the new tokens behind the sequences' ends.  Every block scans the
// sequences' page needs into shared memory (s_base: fresh pages before each
// sequence; -1 for a sequence that is skipped), looks up the cache row of
// each of its tokens, then copies them as one flat run of 16-byte words.
constexpr int kTokMax = 256;           // tokens per block

__global__ void __launch_bounds__(kThreads)
append_kernel(Pages pg, const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new,
              const int *__restrict__ cu, int *__restrict__ table, const int *__restrict__ lens,
              const int *__restrict__ free_pages, const int *__restrict__ free_count,
              int free_capacity, int *__restrict__ lens_out, int *__restrict__ count_out, int num_seqs, int total,
              int max_pages, int per_block) {
    extern __shared__ int s_base[];
    __shared__ int s_warp[kWarps];
    __shared__ int s_row[kTokMax];
    const int tid = threadIdx.x;
    const int count = good_count(free_count, free_capacity);
    // what sequence s asks for; false: unusable offsets or lengths
    auto ask = [&](int s, int &len, int &n) -> bool {
        const int a = __ldg(cu + s);
        n = __ldg(cu + s + 1) - a;
        len = __ldg(lens + s);
        return a >= 0 && n >= 0 && a <= total - n && len >= 0 && len <= max_pages * kPage - n;
    };
    int running, left;
    // marked: s_base holds -1 for sequences that are left out already; true if an
    // offset descends or leaves [0, total]
    auto plan = [&](bool marked) -> bool {
        bool bad = false;
        running = 0;
        left = INT_MAX;
        for (int s0 = 0; s0 < num_seqs; s0 += kThreads) {
            const int s = s0 + tid;
            int len = 0, n = 0, need = 0;
            bool ok = false;
            if (s < num_seqs) {
                ok = ask(s, len, n) && !(marked && s_base[s] < 0);
                if (ok) {
                    need = pages_of(len + n) - pages_of(len);
                } else {
                    const int a = __ldg(cu + s);
                    bad |= a < 0 || n < 0 || a > total - n;
                    if (blockIdx.x == 0) report_error(kDevErrInput);
                }
            }
            int sum;
            const int base = running + block_scan(need, s_warp, sum);
            running += sum;
            if (s < num_seqs) {
                if (ok && need > 0 && base > count - need) {      // out of pages
                    left = min(left, base);
                    ok = false;
                }
                s_base[s] = ok ? base : -1;
            }
        }
        return bad;
    };
    const bool unsorted = __syncthreads_or(plan(false));
    if (unsorted) {
        // the sequences whose tokens lie behind those of the ones before are
        // appended to, the others are left out
        if (tid == 0) {
            int end = 0;
            for (int s = 0; s < num_seqs; ++s) {
                const int a = __ldg(cu + s), e = __ldg(cu + s + 1);
                const bool good = a >= end && e >= a && e <= total;
                s_base[s] = good ? 0 : -1;
                if (good) end = e;
            }
        }
        __syncthreads();
        plan(true);
        __syncthreads();
    }
    if (left != INT_MAX && blockIdx.x == 0) report_error(kDevErrPages);
    // pages handed out: all, or those before the first sequence left out
    left = __reduce_min_sync(0xffffffffu, left);
    if (lane_id() == 0) s_warp[warp_id()] = left;
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) {
        for (int w = 0; w < kWarps; ++w) running = min(running, s_warp[w]);
        *count_out = count - running;
    }
    // tables and lengths of every gridDim.x-th sequence
    for (int s = blockIdx.x; s < num_seqs; s += gridDim.x) {
        int len, n;
        ask(s, len, n);
        const int base = s_base[s];
        bool add = base >= 0;
        if (add && n > 0) {
            // the pages its tokens go to must exist, or it is left out
            const int used = pages_of(len), used_new = pages_of(len + n);
            const int *page = free_pages + count - 1 - base + used;
            bool bad = false;
            if (tid == 0 && len % kPage) bad = !exists(pg, __ldcg(table + (size_t)s * max_pages + used - 1));
            for (int c = used + tid; c < used_new; c += kThreads) bad |= !exists(pg, __ldg(page - c));
            add = !__syncthreads_or(bad);
            for (int c = used + tid; add && c < used_new; c += kThreads)
                table[(size_t)s * max_pages + c] = __ldg(page - c);
            if (!add && tid == 0) report_error(kDevErrInput);
        }
        if (tid == 0) lens_out[s] = add ? len + n : len;
    }
    const int t0 = blockIdx.x * per_block, nt = min(per_block, total - t0);
    if (nt <= 0) return;
    for (int i = tid; i < nt; i += kThreads) {
        const int t = t0 + i;
        int lo = 0, hi = num_seqs;          // the last s with cu[s] <= t
        if (unsorted)                       // (of those not left out)
            for (int s = 0; s < num_seqs; ++s)
                if (s_base[s] >= 0 && __ldg(cu + s) <= t) lo = s;
        while (!unsorted && hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(cu + mid) <= t) lo = mid; else hi = mid;
        }
        int row = -1, len, n;
        if (ask(lo, len, n) && s_base[lo] >= 0 && t >= __ldg(cu + lo) && t - __ldg(cu + lo) < n) {
            const int pos = len + t - __ldg(cu + lo), c = pos / kPage, used = pages_of(len);
            // (entries below `used` are not written by this launch)
            const int page = c < used ? __ldcg(table + (size_t)lo * max_pages + c)
                                      : __ldg(free_pages + count - 1 - (s_base[lo] + c - used));
            if (exists(pg, page)) row = page * kPage + pos % kPage;
            else report_error(kDevErrInput);
        }
        s_row[i] = row;
    }
    __syncthreads();
    const int words = nt * pg.tok16;
    const size_t src0 = (size_t)t0 * pg.tok16;
    constexpr int U = 4;
    for (int i = tid; i < words; i += U * kThreads) {
        uint4 a[U], b[U];
        size_t to[U];
        #pragma unroll
        for (int u = 0; u < U; ++u) {
            const int w = i + u * kThreads;
            to[u] = ~(size_t)0;
            if (w < words) {
                const int tok = w / pg.tok16, row = s_row[tok];
                if (row >= 0) to[u] = (size_t)row * pg.tok16 + (w - tok * pg.tok16);
                a[u] = __ldcs(k_new + src0 + w);
                b[u] = __ldcs(v_new + src0 + w);
            }
        }
        #pragma unroll
        for (int u = 0; u < U; ++u)
            if (to[u] != ~(size_t)0) {
                __stcs(pg.k + to[u], a[u]);
                __stcs(pg.v + to[u], b[u]);
            }
    }
}

// -------------------------------------------------------- the pages in use
// One bit per page, set if a used table entry names it.  The bitmap is
// cleared before.  Grid: (pieces of a row, sequences).
constexpr int kMarkSpan = 4 * kThreads;

__global__ void __launch_bounds__(kThreads)
mark_kernel(const int *__restrict__ table, const int *__restrict__ lens, uint32_t *__restrict__ bits,
            int max_pages, int num_pages) {
    const int s = blockIdx.y;
    const int used = pages_of(good_len(__ldg(lens + s), max_pages));
    const int c0 = blockIdx.x * kMarkSpan;
    #pragma unroll
    for (int u = 0; u < kMarkSpan / kThreads; ++u) {
        const int c = c0 + u * kThreads + threadIdx.x;
        if (c >= used) break;
        const int page = __ldg(table + (size_t)s * max_pages + c);
        if (page < 0 || page >= num_pages) {
            report_error(kDevErrInput);
            continue;
        }
        const uint32_t bit = 1u << (page & 31);
        if (!(__ldcg(bits + (page >> 5)) & bit)) atomicOr(bits + (page >> 5), bit);
    }
}

// The pages of word w that exist.
__device__ __forceinline__ uint32_t page_mask(int w, int num_pages) {
    const int n = num_pages - w * 32;
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// free_pages: the pages not in use, highest first, so that the lowest is at
// the end and handed out first.  One word (32 pages) per thread; a page's
// index is the number of free pages above it.
__global__ void __launch_bounds__(kThreads)
collect_kernel(const uint32_t *__restrict__ bits, int *__restrict__ free_pages,
               int *__restrict__ free_count, int num_pages) {
    __shared__ int s_warp[kWarps];
    const int words = (num_pages + 31) / 32;
    const int w = blockIdx.x * kThreads + threadIdx.x;
    int above = 0;
    for (int i = (blockIdx.x + 1) * kThreads + threadIdx.x; i < words; i += kThreads)
        above += __popc(~__ldg(bits + i) & page_mask(i, num_pages));
    above = block_sum(above, s_warp);
    const uint32_t mine = w < words ? ~__ldg(bits + w) & page_mask(w, num_pages) : 0u;
    int total;
    const int before = block_scan(__popc(mine), s_warp, total);
    const int top = above + total - before - __popc(mine);   // free pages above this word
    // a warp writes its 32 words one after the other, a lane per page
    const int lane = lane_id();
    for (int i = 0; i < 32; ++i) {
        const uint32_t m = __shfl_sync(0xffffffffu, mine, i);
        const int t = __shfl_sync(0xffffffffu, top, i);
        const int page = (blockIdx.x * kThreads + warp_id() * 32 + i) * 32 + lane;
        if (m >> lane & 1) free_pages[t + __popc(m & ~((2u << lane) - 1u))] = page;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *free_count = above + total;
}

// Compaction's plan.  n_live pages are in use; the i-th used page at or above
// n_live goes to the i-th free page below it.  from[i], to[i]: the moves;
// rank[p]: the move of page p.  The free list afterwards is num_pages - 1
// down to n_live.
__global__ void __launch_bounds__(kThreads)
compact_plan_kernel(const uint32_t *__restrict__ bits, int *__restrict__ from, int *__restrict__ to,
                    int *__restrict__ rank, int *__restrict__ header, int *__restrict__ free_pages,
                    int *__restrict__ free_count, int num_pages) {
    __shared__ int s_warp[kWarps];
    const int words = (num_pages + 31) / 32;
    const int w0 = blockIdx.x * kThreads, w = w0 + threadIdx.x;
    int live = 0, below = 0;
    for (int i = threadIdx.x; i < words; i += kThreads) {
        const int c = __popc(__ldg(bits + i));
        live += c;
        if (i < w0) below += c;
    }
    live = block_sum(live, s_warp);
    below = block_sum(below, s_warp);
    int kept = 0;                          // used pages below n_live: they stay
    for (int i = threadIdx.x; i * 32 < live; i += kThreads)
        kept += __popc(__ldg(bits + i) & page_mask(i, live));
    kept = block_sum(kept, s_warp);
    const uint32_t mine = w < words ? __ldg(bits + w) : 0u;
    int total;
    const int before = below + block_scan(__popc(mine), s_warp, total);   // used pages below word w
    const int lane = lane_id();
    for (int i = 0; i < 32; ++i) {
        const uint32_t m = __shfl_sync(0xffffffffu, mine, i);
        const int b = __shfl_sync(0xffffffffu, before, i);
        const int page = (w0 + warp_id() * 32 + i) * 32 + lane;
        if (page >= num_pages) continue;
        const int lower = b + __popc(m & ((1u << lane) - 1u));
        const bool used = m >> lane & 1;
        if (used && page >= live) {
            from[lower - kept] = page;
            rank[page] = lower - kept;
        } else if (!used && page < live) {
            to[page - lower] = page;
        }
        if (page >= live) free_pages[num_pages - 1 - page] = page;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *free_count = num_pages - live;
        header[0] = live;
        header[1] = live - kept;
    }
}

// Compaction's moves (sources lie at or above n_live, destinations below, so
// their order does not matter), and the renamed tables.
__global__ void __launch_bounds__(kThreads)
compact_move_kernel(Pages pg, const int *table, int *table_out, const int *__restrict__ lens,
                    const int *__restrict__ from, const int *__restrict__ to,
                    const int *__restrict__ rank, const int *__restrict__ header, int num_seqs,
                    int max_pages) {
    const int live = __ldg(header), moves = __ldg(header + 1);
    for (int s = blockIdx.x; s < num_seqs; s += gridDim.x) {
        const int used = pages_of(good_len(__ldg(lens + s), max_pages));
        for (int c = threadIdx.x; c < used; c += kThreads) {
            const size_t i = (size_t)s * max_pages + c;
            const int page = table[i];
            table_out[i] = (page >= live && page < pg.num_pages) ? __ldg(to + __ldg(rank + page)) : page;
        }
    }
    // half a page (K or V) at a time
    for (int m = blockIdx.x; m < 2 * moves; m += gridDim.x)
        copy_page(pg, __ldg(from + (m >> 1)), __ldg(to + (m >> 1)), kPage, !(m & 1), m & 1);
}

// ------------------------------------------------------------------- copy
// Page src[i] to page dst[i].  An entry whose destination is also the source
// of an entry, or the destination of a later one, is left out and reported,
// so no block reads or writes a page that another writes.  A block takes
// kCopyEntries entries and compares them with the whole list.
constexpr int kCopyEntries = 4;

__global__ void __launch_bounds__(kThreads)
copy_pages_kernel(Pages pg, const int *__restrict__ src, const int *__restrict__ dst, int n) {
    __shared__ int s_bad[kCopyEntries];
    const int e0 = blockIdx.x * kCopyEntries;
    if (threadIdx.x < kCopyEntries) s_bad[threadIdx.x] = 0;
    __syncthreads();
    int d[kCopyEntries], bad[kCopyEntries];
    #pragma unroll
    for (int u = 0; u < kCopyEntries; ++u) {
        d[u] = e0 + u < n ? __ldg(dst + e0 + u) : -1;
        bad[u] = 0;
    }
    for (int j = threadIdx.x; j < n; j += kThreads) {
        const int sj = __ldg(src + j), dj = __ldg(dst + j);
        if (sj < 0 || dj < 0 || sj >= pg.num_pages || dj >= pg.num_pages) continue;
        #pragma unroll
        for (int u = 0; u < kCopyEntries; ++u)
            bad[u] |= (sj == d[u] && j != e0 + u) | (dj == d[u] && j > e0 + u);
    }
    #pragma unroll
    for (int u = 0; u < kCopyEntries; ++u)
        if (bad[u]) s_bad[u] = 1;
    __syncthreads();
    for (int u = 0; u < kCopyEntries && e0 + u < n; ++u) {
        const int s = __ldg(src + e0 + u), t = d[u];
        if (s == -1 && t == -1) continue;                  // an unused entry
        if (s < 0 || t < 0 || s >= pg.num_pages || t >= pg.num_pages || s_bad[u]) {
            if (threadIdx.x == 0) report_error(kDevErrInput);
            continue;
        }
        if (s != t) copy_page(pg, s, t, kPage, true, true);
    }
}

Pages make_pages(const CachePages &c) {
    Pages pg;
    pg.k = static_cast<uint4 *>(c.k);
    pg.v = static_cast<uint4 *>(c.v);
    pg.ks = c.k_scale;
    pg.vs = c.v_scale;
    pg.num_pages = c.num_pages;
    pg.Hkv = c.Hkv;
    pg.tok16 = (int)((long long)c.Hkv * c.d * c.elem_bytes / 16);
    return pg;
}

int launched() { return cudaGetLastError() == cudaSuccess ? 0 : -5; }

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Clears the bitmap at the workspace's start and marks the pages in use.
int mark_pages(const int *table, const int *lens, int num_seqs, int max_pages, int num_pages,
               uint32_t *bits, cudaStream_t stream) {
    if (cudaMemsetAsync(bits, 0, (size_t)(num_pages + 31) / 32 * 4, stream) != cudaSuccess) return -5;
    if (num_seqs == 0) return 0;
    const dim3 grid((unsigned)((max_pages + kMarkSpan - 1) / kMarkSpan), (unsigned)num_seqs);
    mark_kernel<<<grid, kThreads, 0, stream>>>(table, lens, bits, max_pages, num_pages);
    return launched();
}

}  // namespace cache_impl

using namespace cache_impl;

int launch_cache_fork(const CachePages &c, const int *table, const int *lens, int slots_in,
                      const int *parents, int slots_out, const int *free_pages,
                      const int *free_count, int free_capacity, int *table_out, int *lens_out,
                      int *count_out, int max_pages, cudaStream_t stream) {
    // a slot or a few per block, about four blocks per SM
    const int want = 2 * device_sm_count();
    const int per = slots_out > want ? (slots_out + want - 1) / want : 1;
    const int blocks = slots_out > 0 ? (slots_out + per - 1) / per : 1;
    fork_kernel<<<dim3(blocks, 2), kThreads, (size_t)slots_in * sizeof(int), stream>>>(
        make_pages(c), table, lens, parents, free_pages, free_count, free_capacity, table_out, lens_out,
        count_out, slots_in, slots_out, max_pages, per);
    return launched();
}

int launch_cache_append(const CachePages &c, const void *k_new, const void *v_new, const int *cu,
                        int num_seqs, int total, int *table, const int *lens,
                        const int *free_pages, const int *free_count, int free_capacity,
                        int *lens_out, int *count_out, int max_pages, cudaStream_t stream) {
    const int want = 4 * device_sm_count();
    int per = (total + want - 1) / want;
    per = per < 1 ? 1 : per > kTokMax ? kTokMax : per;
    const int blocks = total > 0 ? (total + per - 1) / per : 1;
    append_kernel<<<blocks, kThreads, (size_t)num_seqs * sizeof(int), stream>>>(
        make_pages(c), static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new), cu,
        table, lens, free_pages, free_count, free_capacity, lens_out, count_out, num_seqs, total,
        max_pages, per);
    return launched();
}

int launch_cache_copy(const CachePages &c, const int *src, const int *dst, int n,
                      cudaStream_t stream) {
    copy_pages_kernel<<<(n + kCopyEntries - 1) / kCopyEntries, kThreads, 0, stream>>>(make_pages(c),
                                                                                     src, dst, n);
    return launched();
}

size_t cache_collect_workspace_bytes(int num_pages) {
    return num_pages <= 0 ? 0 : up256((size_t)(num_pages + 31) / 32 * 4);
}

int launch_cache_collect(const int *table, const int *lens, int num_seqs, int max_pages,
                         int num_pages, int *free_pages, int *free_count, void *workspace,
                         cudaStream_t stream) {
    uint32_t *bits = static_cast<uint32_t *>(workspace);
    const int rc = mark_pages(table, lens, num_seqs, max_pages, num_pages, bits, stream);
    if (rc) return rc;
    const int words = (num_pages + 31) / 32;
    collect_kernel<<<(words + kThreads - 1) / kThreads, kThreads, 0, stream>>>(bits, free_pages,
                                                                              free_count, num_pages);
    return launched();
}

// bitmap | header | from | to | rank
size_t cache_compact_workspace_bytes(int num_pages) {
    return num_pages <= 0 ? 0 : cache_collect_workspace_bytes(num_pages) + 256 +
                                    3 * up256((size_t)num_pages * sizeof(int));
}

int launch_cache_compact(const CachePages &c, const int *table, const int *lens, int num_seqs,
                         int max_pages, int *table_out, int *free_pages, int *free_count,
                         void *workspace, cudaStream_t stream) {
    char *ws = static_cast<char *>(workspace);
    uint32_t *bits = reinterpret_cast<uint32_t *>(ws);
    int *header = reinterpret_cast<int *>(ws + cache_collect_workspace_bytes(c.num_pages));
    const size_t step = up256((size_t)c.num_pages * sizeof(int)) / sizeof(int);
    int *from = header + 64, *to = from + step, *rank = to + step;
    int rc = mark_pages(table, lens, num_seqs, max_pages, c.num_pages, bits, stream);
    if (rc) return rc;
    const int words = (c.num_pages + 31) / 32;
    compact_plan_kernel<<<(words + kThreads - 1) / kThreads, kThreads, 0, stream>>>(
        bits, from, to, rank, header, free_pages, free_count, c.num_pages);
    rc = launched();
    if (rc) return rc;
    compact_move_kernel<<<8 * device_sm_count(), kThreads, 0, stream>>>(
        make_pages(c), table, table_out, lens, from, to, rank, header, num_seqs, max_pages);
    return launched();
}

}  // namespace fa
