// shared_sm100.cu -- attention of many query rows to one set of keys, split
// over the keys: decode of a batch whose sequences share a prefix, and decode
// against an encoder's states.
//
// What it computes: O = softmax(Q K^T * scale) V and LSE of every query row,
// all keys visible up to a length.  The softmax over several sets of keys
// r = 1, 2, ... (the shared pages, the sequence's own pages, pieces of
// either) is joined from the sets' own results:
//     M = max_r LSE_r,  O = sum_r 2^(LSE_r - M) O_r / sum_r 2^(LSE_r - M).
//
// How:
//   * The work is a list of items.  An item is up to 256 query rows and the
//     keys they all see: the rows (sequence, head of the KV head's group) of a
//     group of sequences on the group's shared pages, so that these cross HBM
//     once and not once per sequence; the group's heads of one sequence on
//     the sequence's own pages; the tokens and heads of one sequence on its
//     encoder states.  All items exist once per KV head.
//   * Every KV head gets the same number n of CTAs (n * Hkv of the SMs), and
//     each of them an equal share of the items' key blocks, cut anywhere:
//     with lengths from one token to many thousand every SM still ends at the
//     same time.  CTAs of the KV heads at the same place read the same tokens
//     at the same time, so that whole token rows cross HBM together.  A share
//     gives one partial (fp32 O, LSE) per row and item it touches.  The plan
//     (prefix sums over the items) is computed by every CTA for itself in
//     shared memory, about two microseconds; lengths never come to the host.
//   * Warps 8 and 10 feed a ring of K and V tiles (128 keys) by TMA, page by
//     page through the block table, and run ahead over the items.  V rows
//     behind a sequence's end are cleared (they may hold anything, and P = 0
//     times NaN is NaN).
//   * Up to 32 rows (a sequence's own pages, a token against its encoder
//     states): S^T = K Q^T and O^T += V^T P^T, so that the keys (then the head
//     dim) fill the 128 lanes of the products and N is 16 or 32.  Warp 9
//     issues S^T up to four blocks ahead, warp 11 O^T.  A softmax thread has
//     one key and all rows; P^T goes through shared memory.  The two softmax
//     warpgroups take the shares in turn, so that one starts the next while
//     the other still finishes its own.
//   * More rows: S = Q K^T and O += P V as in the prefill, P in tensor memory,
//     warp 9 issuing both.  More than 128 rows: each warpgroup has a tile of
//     128 rows and sees every block.  Up to 128: both have the same rows and
//     take the blocks in turn; their results are joined through shared memory.
//     Up to 64: the rows stand twice in the tile's 128 lanes, each copy takes
//     half of a block's keys (P = 0 in the other's), and four warps share the
//     exponentials instead of two.
//   * shared_combine_kernel joins the partials of each row.
#include <climits>
#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {

namespace shared_impl {

constexpr int kPage = 16;           // tokens per cache page
constexpr int kBlockM = 128;        // rows per tile (TMEM lanes)
constexpr int kBlockN = 128;        // keys per K/V tile
constexpr int kPagesPerBlock = kBlockN / kPage;
constexpr int kRows = 2 * kBlockM;  // rows per item
constexpr int kThreads = 384;
constexpr int kWarpK = 8, kWarpMma = 9, kWarpV = 10;   // and 11: P V of few rows
// Registers: launched with 384 x 168; softmax warpgroups 216, the rest 72
// (2 * 128 * 216 + 128 * 72 = 64,512).
constexpr int kRegsSoftmax = 216, kRegsControl = 72;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsControl <= kThreads * 168, "register split");
constexpr float kRescaleThreshold = 8.0f;   // log2 units, as in the prefill
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxSeqs = kSharedMaxSeqs;    // sequences per launch
constexpr int kMaxGroupItems = 1024;        // group <= 128 heads: at most S/2 + S/2 items
constexpr int kMaxItems = kSharedMaxItems;
static_assert(kMaxSeqs + kMaxGroupItems <= kMaxItems, "items of a paged batch");
constexpr int kFewRows = 32;                // rows at most in the transposed form
constexpr int kSBufs = 4;                   // S^T buffers per warpgroup, 32 columns each
// What a key block costs a CTA, by the item's rows, and an item besides (its
// first loads and its epilogue).  Measured on prefixes of 131,072 tokens, 8 KV
// heads, us per block: d = 128 1.32 (4 rows), 1.35 (32), 1.33 to 1.41 (36 to
// 128), 2.09 (132), 2.16 (192), 2.27 (256); d = 64 0.81 (4), 0.86 (16), 1.02
// (32), 0.99 (36), 1.11 (64), 1.17 to 1.24 (68 to 96), 1.47 (128), 2.33 (132),
// 2.37 (192), 2.64 (256).  Up to 128 rows at d = 128 that is the rate of HBM,
// 6.7 to 7.2 TB/s.
template <int D>
struct Cost {
    static constexpr int kFew = 3, kOne = D == 128 ? 3 : 4, kPair = D == 128 ? 5 : 8;
};
constexpr int kCostItem = 1, kCostBigItem = 5;

template <int D>
struct Cfg {
    static constexpr int kBoxes = D / 64;
    static constexpr int kBoxBytes = kBlockM * 128;            // 128 rows x 128 bytes
    static constexpr int kTileBytes = kBlockM * D * 2;
    static constexpr int kStages = D == 128 ? 4 : 8;           // K in the even slots, V in the odd
    // Q of a warpgroup's tile: 32 KB for either head dim.  With few rows: two
    // buffers of Q and two of P^T.
    static constexpr int kQBytes = 32768;
    static constexpr int kOffKV = 2 * kQBytes;
    static constexpr int kOffTable = kOffKV + kStages * kTileBytes;
    static constexpr uint32_t kColO = 256;                     // O_t at 256 + t*D
    static constexpr int kChunk = 32;                          // columns joined at a time
};

// The plan, in shared memory.
constexpr int kSlotBits = 20;
static_assert(kRows * (kMaxItems + kSharedMaxCtas) < 1 << kSlotBits && kMaxItems < 1 << (32 - kSlotBits),
              "partial rows and items in a word");
struct Table {
    int start[kMaxItems + 1];        // cost before the item; INT_MAX behind the last
    // partial rows before the item, and from kSlotBits on how many items on the next
    // one with keys (or the end) is
    uint32_t slot[kMaxItems];
    uint32_t some[kMaxItems / 32];   // a bit per item: it has keys
    uint32_t gi[kMaxGroupItems];     // group items: group | row pair << 16
    uint16_t cu[kMaxSeqs + 2];       // first sequence of each group
    int own[kMaxSeqs];               // pages of each sequence that its group reads
    int keys[kMaxSeqs];              // keys behind them (not paged: all keys)
    int num_group_items, num_items, span;
    int first;                       // this CTA's first item << 8 | share of it (INT_MAX: none)
};
static_assert(kSharedMaxCtas <= 256, "shares of an item in 8 bits");

struct Params {
    const uint16_t *q;
    const int *block_table, *lens, *cu_groups, *prefix_lens;
    float *part_o, *part_lse;  // [Hkv][cap][D], [Hkv][cap], log2 units
    int4 *items;               // {slot, partials, rows, -}
    int4 *seqs;                // {own item, first group item or -1, group's first sequence, -}
    int S, num_groups, num_pages, max_pages;
    int Hq, Hkv, G, Nq, Nk, pairs;
    uint32_t G_magic;
    int n;                     // CTAs per KV head
    int cost_few, cost_one, cost_pair;
    int total_k;               // dense: stored key rows
    long long cap;
    float scale_log2;
};

struct Shared {
    uint64_t q_full[2];
    // A wait knows a phase by its parity alone.  A warp that skips uses of a slot
    // (an issuer, the V tiles of the other's shares) may wait for a later one only
    // after something that implies that all earlier ones are over.
    uint64_t kv_full[8], kv_empty[8], tail;
    uint64_t s_full[2], p_lo[2], p_hi[2], o_full[2];
    uint64_t st_full[2][kSBufs], st_empty[2][kSBufs], pt_full[2][2], pt_empty[2][2];
    uint64_t drain[2];
    float2 ml[8][32];
    int scan[kThreads / 32];
    uint32_t tmem_base;
    int abort;
};

// Rows of a P^T buffer (and N of the transposed products): 16 or 32.
__device__ __forceinline__ int few_n(int rows) { return rows <= 16 ? 16 : 32; }

// Within a warpgroup's Q tile: P^T buffer b, and Q buffer b (its second box
// one kBoxBytes on).
__device__ __forceinline__ int few_p(int b) { return b ? 20480 : 4096; }
__device__ __forceinline__ int few_q(int b) { return b * 12288; }

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// A sequence's length.  One that its table cannot hold is clamped; one that its
// stored keys cannot hold counts as none, and the combine leaves its rows alone.
template <bool PAGED>
__device__ __forceinline__ int good_length(const Params &p, int L) {
    const int most = PAGED ? p.max_pages * kPage : p.Nk;
    if (L < 0 || L > most) {
        if (blockIdx.x == 0) report_error(kDevErrInput);
        L = L < 0 || !PAGED ? 0 : most;
    }
    return L;
}

// One item: which rows, which keys.
struct Item {
    int tok0;        // token of row 0 of the rows' set
    int row0, rows;  // the item's rows of that set
    int src;         // sequence whose block table (or key rows) it reads
    int page0;       // paged: first page
    int keys;
};

template <bool PAGED>
__device__ __forceinline__ Item get_item(const Params &p, const Table &tab, int groups, int i) {
    Item w;
    int all = p.Nq * p.G;
    w.row0 = 0;
    w.page0 = 0;
    if constexpr (PAGED) {
        if (i < groups) {
            const int g = tab.gi[i] & 0xffff, first = tab.cu[g];
            w.tok0 = w.src = first;
            all = (tab.cu[g + 1] - first) * p.G;
            w.row0 = (int)(tab.gi[i] >> 16) * kRows;
            w.keys = tab.own[first] * kPage;
        } else {
            w.tok0 = w.src = i - groups;
            w.page0 = tab.own[w.src];
            w.keys = tab.keys[w.src];
        }
    } else {
        w.src = p.pairs == 1 ? i : i / p.pairs;
        w.tok0 = w.src * p.Nq;
        w.row0 = (i - w.src * p.pairs) * kRows;
        w.keys = tab.keys[w.src];
    }
    w.rows = min(kRows, all - w.row0);
    return w;
}

// x / G for the rows of a launch (G_magic = ceil(2^32 / G), exact as x * G < 2^32).
__device__ __forceinline__ int div_group(const Params &p, int x) {
    return p.G == 1 ? x : (int)__umulhi((uint32_t)x, p.G_magic);
}

// ceil(x / c) for the costs, x < 2^30.
__device__ __forceinline__ int div_cost(int x, int c) {
    const uint32_t y = (uint32_t)(x + c - 1);
    return (int)(c == 3 ? __umulhi(y, 0x55555556u) : c == 5 ? __umulhi(y, 0x33333334u)
                 : c == 4 ? y >> 2 : y >> 3);
}

__device__ __forceinline__ int block_cost(const Params &p, int rows) {
    return rows > kBlockM ? p.cost_pair : rows > 16 ? p.cost_one : p.cost_few;
}
__device__ __forceinline__ int item_cost(const Params &p, int rows, int keys) {
    return keys > 0 ? ceil_div(keys, kBlockN) * block_cost(p, rows) + (rows > kFewRows ? kCostBigItem : kCostItem)
                    : 0;
}

// x / span, 0 <= x < 2^31, given inv = floor((2^32 - 1) / span).
__device__ __forceinline__ int div_span(int x, int span, uint32_t inv) {
    const int q = (int)__umulhi((uint32_t)x, inv);
    return x - q * span >= span ? q + 1 : q;
}

// Exclusive prefix sum over the block's threads; `total` gets the sum.
__device__ __forceinline__ int block_scan(int x, int *s_warp, int &total) {
    const int lane = lane_id(), warp = warp_id();
    int inc = x;
    #pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    const int sum = lane < kThreads / 32 ? s_warp[lane] : 0;
    total = __reduce_add_sync(0xffffffffu, sum);
    return __reduce_add_sync(0xffffffffu, lane < warp ? sum : 0) + inc - x;
}

// The group of sequence s, or -1.
__device__ __forceinline__ int group_of(const int *cu, int ng, int s) {
    int lo = 0, hi = ng;
    #pragma unroll 1
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= s) lo = mid; else hi = mid;
    }
    return ng > 0 && cu[lo] <= s && s < cu[lo + 1] ? lo : -1;
}

// All threads of the block; ends with a barrier.  `scratch`: room for
// 3 * kMaxSeqs + 1 ints.  Everything read from global memory is asked for at
// once, so that the plan costs one latency and some barriers.
template <bool PAGED>
__device__ void make_plan(const Params &p, Table &tab, int *scratch, int *s_warp) {
    const int tid = threadIdx.x;
    const bool lead = blockIdx.x == 0;
    int ni = 0, ng = PAGED ? p.num_groups : 0;
    int *cu = scratch, *least = cu + kMaxSeqs + 1, *prefix = least + kMaxSeqs;
    if (PAGED && ng > 0) {
        #pragma unroll 1
        for (int g = tid; g <= ng; g += kThreads) {
            cu[g] = __ldg(p.cu_groups + g);
            if (g < ng) {
                prefix[g] = __ldg(p.prefix_lens + g);
                least[g] = INT_MAX;
            }
        }
    }
    #pragma unroll 1
    for (int s = tid; s < p.S; s += kThreads) {
        tab.keys[s] = good_length<PAGED>(p, p.lens ? __ldg(p.lens + s) : p.Nk);
        tab.own[s] = 0;
    }
    if (PAGED && ng > 0) {
        __syncthreads();
        bool bad = false;
        #pragma unroll 1
        for (int g = tid; g < ng; g += kThreads)
            bad |= cu[g] < 0 || cu[g + 1] < cu[g] || cu[g + 1] > p.S;
        if (__syncthreads_or(bad)) {       // unusable groups: every sequence by itself
            if (lead && tid == 0) report_error(kDevErrInput);
            ng = 0;
        }
        // no more is shared than the group's shortest sequence has
        #pragma unroll 1
        for (int s = tid; s < p.S; s += kThreads) {
            const int g = group_of(cu, ng, s);
            if (g >= 0) atomicMin(&least[g], tab.keys[s]);
        }
        __syncthreads();
        #pragma unroll 1
        for (int g0 = 0; g0 < ng; g0 += kThreads) {
            const int g = g0 + tid;
            int items = 0, pages = 0;
            if (g < ng) {
                int len = prefix[g];
                if (len < 0) {
                    if (lead) report_error(kDevErrInput);
                    len = 0;
                }
                const int cnt = cu[g + 1] - cu[g];
                if (cnt >= 2) pages = min(len, least[g]) / kPage;
                if (pages > 0) items = ceil_div(cnt * p.G, kRows);
            }
            int total;
            const int base = ni + block_scan(items, s_warp, total);
            ni += total;
            if (g < ng) {
                least[g] = pages;
                prefix[g] = pages > 0 ? base : -1;       // now the group's first item
                tab.cu[g] = (uint16_t)cu[g];
                if (g == ng - 1) tab.cu[ng] = (uint16_t)cu[ng];
                #pragma unroll 1
                for (int r = 0; r < items; ++r) tab.gi[base + r] = (uint32_t)g | (uint32_t)r << 16;
            }
        }
        __syncthreads();
        #pragma unroll 1
        for (int s = tid; s < p.S; s += kThreads) {
            const int g = group_of(cu, ng, s), pages = g >= 0 ? least[g] : 0;
            tab.own[s] = pages;
            tab.keys[s] -= pages * kPage;
            if (lead) p.seqs[s] = make_int4(ni + s, g >= 0 ? prefix[g] : -1, g >= 0 ? cu[g] : 0, 0);
        }
    } else if (PAGED && lead) {
        #pragma unroll 1
        for (int s = tid; s < p.S; s += kThreads) p.seqs[s] = make_int4(s, -1, 0, 0);
    }
    const int N = PAGED ? ni + p.S : p.S * p.pairs;
    if (tid == 0) {
        tab.num_group_items = ni;
        tab.num_items = N;
        tab.first = INT_MAX;
        tab.start[N] = INT_MAX;
    }
    if (tid < kMaxItems / 32) tab.some[tid] = 0;
    __syncthreads();
    // cost before each item; a thread has `per` consecutive ones
    const int per = ceil_div(N, kThreads), i0 = min(N, tid * per), i1 = min(N, i0 + per);
    int sum = 0, total;
    #pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const Item w = get_item<PAGED>(p, tab, ni, i);
        tab.start[i] = sum;
        sum += item_cost(p, w.rows, w.keys);
    }
    const int before = block_scan(sum, s_warp, total);
    // (every share must hold the start of a block of any item it lies inside:
    // no block costs more than a share; only batches of more than 128 rows can
    // have the dearest kind)
    const int most = p.S * p.Nq * p.G > kBlockM ? p.cost_pair : p.cost_one;
    const int span = max(most, ceil_div(total, p.n));
    const uint32_t inv = 0xffffffffu / (uint32_t)span;
    const int share = blockIdx.x / p.Hkv, lo = share * span;
    int rows = 0;
    #pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const Item w = get_item<PAGED>(p, tab, ni, i);
        const int start = tab.start[i] + before;
        tab.start[i] = start;
        int parts = 0;
        if (w.keys > 0) {
            atomicOr(&tab.some[i >> 5], 1u << (i & 31));
            const int last = start + (ceil_div(w.keys, kBlockN) - 1) * block_cost(p, w.rows);
            const int s0 = div_span(start, span, inv);
            parts = div_span(last, span, inv) - s0 + 1;
            if (last >= lo && start < lo + span) atomicMin(&tab.first, i << 8 | (share - s0));
        }
        tab.slot[i] = (uint32_t)rows;
        if (lead) p.items[i] = make_int4(0, parts, w.rows, 0);
        rows += parts * w.rows;
    }
    int all;
    const int slot0 = block_scan(rows, s_warp, all);
    #pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const int slot = (int)tab.slot[i] + slot0;
        if (lead) p.items[i].x = slot;
        int next = i + 1;
        uint32_t later = next < N ? tab.some[next >> 5] >> (next & 31) : 1u;
        #pragma unroll 1
        while (!later) {
            next = (next | 31) + 1;
            later = next < N ? tab.some[next >> 5] : 1u;
        }
        next = min(N, next + __ffs(later) - 1);
        tab.slot[i] = (uint32_t)slot | (uint32_t)(next - i) << kSlotBits;
    }
    if (tid == 0) tab.span = span;
    __syncthreads();
}

// One CTA's share of an item.
struct Work {
    Item it;
    int kb0, kb1;    // key blocks
    bool few;        // transposed form, by warpgroup `wg`
    int wg;
    int rep;         // copies of the rows in a tile's lanes
    bool pair;       // two row tiles on every block (else: one, blocks in turn)
    int slot;        // first partial row
    uint32_t ring;   // ring position of its first K tile
};

struct Walker {
    int i, lo, hi, groups, turn;
    int part;       // of the first item, whose blocks may begin before lo; 0 of the others
    uint32_t ring;
    __device__ __forceinline__ void begin(const Params &p, const Table &tab) {
        turn = 0;
        ring = 0;
        groups = tab.num_group_items;
        lo = blockIdx.x / p.Hkv * tab.span;
        hi = lo + tab.span;
        i = min(tab.first >> 8, tab.num_items);
        part = tab.first & 255;
    }
    template <bool PAGED>
    __device__ __forceinline__ bool next(const Params &p, const Table &tab, Work &w) {
        // (the plan says which item with keys comes next: no loop here over those without)
        const int start = tab.start[i];
        if (start >= hi) return false;
        const uint32_t slot = tab.slot[i];
        w.it = get_item<PAGED>(p, tab, groups, i);
        const int cost = block_cost(p, w.it.rows), nb = ceil_div(w.it.keys, kBlockN);
        w.kb0 = start >= lo ? 0 : min(nb, div_cost(lo - start, cost));
        w.kb1 = min(nb, div_cost(hi - start, cost));
        w.slot = (int)(slot & ((1u << kSlotBits) - 1u)) + part * w.it.rows;
        i += slot >> kSlotBits;
        part = 0;
        w.pair = w.it.rows > kBlockM;
        w.few = w.it.rows <= kFewRows;
        w.wg = turn;
        if (w.few) turn ^= 1;
        w.rep = w.it.rows > 64 ? 1 : 2;
        w.ring = ring;
        ring += 2 * (w.kb1 - w.kb0);
        return true;
    }
};

// Whether V rows behind the item's last key have to be cleared: what the slot
// or the page held (paged), what lies behind the sequence (dense; rows past the
// tensor arrive as zeros).
template <bool PAGED>
__device__ __forceinline__ bool needs_clear(const Params &p, const Work &w, int valid) {
    return valid < kBlockN && (PAGED || (long long)w.it.src * p.Nk + w.it.keys < p.total_k);
}

// ------------------------------------------------------------ TMA producers
// Warp 8 fetches K tiles, warp 10 V tiles: a paged tile is 16 (d = 128) small
// copies, some 1,300 cycles to issue, and one warp for both would need the
// whole time in which a block crosses HBM.
// A V tile in which the item's keys end counts its bytes on a barrier of its
// own; the warp waits for them, writes zeros behind the keys and only then
// completes the slot.  It does so after the next tile's copies, or before it
// waits for a slot: the slot may need this very tile.
template <int D, bool PAGED, bool V>
__device__ void producer(const CUtensorMap *tm, const Params &p, const Table &tab, Shared &sh,
                         uint8_t *sKV) {
    using C = Cfg<D>;
    volatile int *abort = &sh.abort;
    const int lane = lane_id(), kvh = blockIdx.x % p.Hkv;
    uint32_t it = V ? 1 : 0;
    int pending = -1, pending_valid = 0;      // slot of a tile to clear
    uint32_t tail_phase = 0;
    auto clear = [&]() -> bool {
        if (!mbar_wait_warp(&sh.tail, tail_phase & 1, abort)) return false;
        ++tail_phase;
        uint8_t *dst = sKV + pending * C::kTileBytes + pending_valid * 128;
        const int words = (kBlockN - pending_valid) * 8;
        for (int b = 0; b < C::kBoxes; ++b)
            for (int i = lane; i < words; i += 32)
                *reinterpret_cast<uint4 *>(dst + b * C::kBoxBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.kv_full[pending]);
        pending = -1;
        return true;
    };
    // lane i < 8: page i of a block (-1: behind the keys)
    auto page_of = [&](const Work &w, int j) -> int {
        const int c = j * kPagesPerBlock + lane;
        if (!PAGED || lane >= kPagesPerBlock || c * kPage >= w.it.keys) return -1;
        return __ldg(p.block_table + (size_t)w.it.src * p.max_pages + w.it.page0 + c);
    };
    Walker walk;
    walk.begin(p, tab);
    Work w, after;
    bool have = walk.next<PAGED>(p, tab, w);
    int j = 0, ahead = -1;
    if (have) {
        j = w.kb0;
        ahead = page_of(w, j);
    }
    while (have) {
        // the pages of the block after this one, of whatever share, are looked
        // up while this one's copies go out
        int page = ahead;
        const bool last = j + 1 == w.kb1;
        if (last) {
            have = walk.next<PAGED>(p, tab, after);
            if (have) ahead = page_of(after, after.kb0);
        } else {
            ahead = page_of(w, j + 1);
        }
        const int valid = w.it.keys - j * kBlockN;
        const int pages = PAGED ? min(kPagesPerBlock, ceil_div(valid, kPage)) : 0;
        if (PAGED && lane < pages && (page < 0 || page >= p.num_pages)) {
            report_error(kDevErrInput);
            page = 0;
        }
        const int slot = it % C::kStages;
        const uint32_t parity = ((it / C::kStages) & 1) ^ 1;
        uint8_t *dst = sKV + slot * C::kTileBytes;
        if (V && pending >= 0 &&
            !__all_sync(0xffffffffu, mbar_test(smem_u32(&sh.kv_empty[slot]), parity)) && !clear())
            goto out;
        if (!mbar_wait_warp(&sh.kv_empty[slot], parity, abort)) goto out;
        const bool tail = V && needs_clear<PAGED>(p, w, valid);
        if (V && tail && pending >= 0 && !clear()) goto out;     // one at a time
        uint64_t *bar = tail ? &sh.tail : &sh.kv_full[slot];
        if (lane == 0)
            mbar_arrive_expect_tx(bar, PAGED ? pages * kPage * D * 2 : C::kTileBytes);
        __syncwarp();
        if (PAGED) {
            if (lane < pages)
                for (int b = 0; b < C::kBoxes; ++b)
                    tma_load_3d(dst + b * C::kBoxBytes + lane * kPage * 128, tm, bar, b * 64, kvh,
                                page * kPage);
        } else if (lane < C::kBoxes) {
            tma_load_3d(dst + lane * C::kBoxBytes, tm, bar, lane * 64, kvh,
                        w.it.src * p.Nk + j * kBlockN);
        }
        __syncwarp();
        if (V && pending >= 0 && !clear()) {
            it += 2;
            goto out;
        }
        if (tail) {
            pending = slot;
            pending_valid = valid;
        }
        it += 2;
        ++j;
        if (last && have) {
            w = after;
            j = w.kb0;
        }
    }
    if (V && pending >= 0) clear();
    return;
out:
    // Leave no copy in flight: wait for the last load issued into each slot.
    if (lane == 0) {
        if (pending >= 0) mbar_drain_wait(&sh.tail, tail_phase & 1);
        for (uint32_t s = V ? 1 : 0; s < C::kStages; s += 2)
            if (it > s && (int)s != pending) mbar_drain_wait(&sh.kv_full[s], ((it - 2 - s) / C::kStages) & 1);
    }
}

// ------------------------------------------------------------ MMA issuers
// Whole warps, of which one lane issues.  Commits cost it some 250 cycles
// each, so there are few: S's, upon which the softmax warps hand the K slot
// back, and that of the V slot.  Products complete in the order of their
// issue, so with S of a tile's next block P V of the block before is done;
// O's own commit comes after a share's last block.  O and the Q tile need no
// barrier of their own: a warpgroup's next Q (and P) arrives only after it
// has read its O.
template <int D, bool PAGED>
__device__ void mma_issuer(const Params &p, const Table &tab, Shared &sh, uint8_t *sQ, uint8_t *sKV) {
    using C = Cfg<D>;
    volatile int *abort = &sh.abort;
    const uint32_t tmem = sh.tmem_base;
    const uint32_t idS = idesc_bf16_f32(kBlockM, kBlockN, false);
    const uint32_t idPV = idesc_bf16_f32(kBlockM, D, true);
    const uint32_t q_lo = desc_lo(smem_u32(sQ), 16), k_lo = desc_lo(smem_u32(sKV), 16);
    const uint32_t v_lo = desc_lo(smem_u32(sKV), C::kBoxBytes);
    constexpr uint32_t kTileStep = C::kTileBytes >> 4, kQStep = C::kQBytes >> 4;
    uint32_t q_uses[2] = {0, 0}, p_cnt[2] = {0, 0}, st_cnt[2] = {0, 0}, fewq[2] = {0, 0};
    // S_t = Q_t K^T (K-major operands, 128-byte swizzle, 64 columns per box)
    auto issue_s = [&](int t, int slot) {
        if (elect_one()) {
            #pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = ((ks >> 2) * C::kBoxBytes + (ks & 3) * 32) >> 4;
                mma_ss_lo(tmem + t * kBlockN, q_lo + t * kQStep + off, k_lo + slot * kTileStep + off,
                          idS, ks > 0 ? 1u : 0u);
            }
            tc_commit(&sh.s_full[t]);
        }
        __syncwarp();
    };
    // O_t += P_t V, keys 0-63 when they are there, then 64-127
    auto issue_pv = [&](int t, int slot, bool &first, bool last, bool free) -> bool {
        #pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (!mbar_wait_warp(half ? &sh.p_hi[t] : &sh.p_lo[t], p_cnt[t] & 1, abort)) return false;
            tc_fence_after();
            if (elect_one()) {
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int ks = half * 4 + k;
                    mma_ts_lo(tmem + C::kColO + t * D, tmem + t * kBlockN + half * 64 + k * 8,
                              v_lo + slot * kTileStep + ((ks * 2048) >> 4), idPV,
                              (ks > 0 || !first) ? 1u : 0u);
                }
                if (half && free) tc_commit(&sh.kv_empty[slot]);
                if (half && last) tc_commit(&sh.o_full[t]);
            }
            __syncwarp();
        }
        ++p_cnt[t];
        first = false;
        return true;
    };
    Walker walk;
    walk.begin(p, tab);
    Work w;
    while (walk.next<PAGED>(p, tab, w)) {
        const int nb = w.kb1 - w.kb0;
        uint32_t it = w.ring;
        if (w.few) {
            // S^T = K Q^T into the warpgroup's next free buffer
            const uint32_t id = idesc_bf16_f32(kBlockN, few_n(w.it.rows), false);
            const uint32_t q = q_lo + w.wg * kQStep + (few_q(fewq[w.wg]++ & 1) >> 4);
            if (!mbar_wait_warp(&sh.q_full[w.wg], q_uses[w.wg] & 1, abort)) goto out;
            ++q_uses[w.wg];
            for (int j = 0; j < nb; ++j, it += 2) {
                const int ks = it % C::kStages;
                const uint32_t n = st_cnt[w.wg]++;
                const int buf = n % kSBufs;
                if (!mbar_wait_warp(&sh.kv_full[ks], (it / C::kStages) & 1, abort)) goto out;
                if (!mbar_wait_warp(&sh.st_empty[w.wg][buf], ((n / kSBufs) & 1) ^ 1, abort)) goto out;
                tc_fence_after();
                if (elect_one()) {
                    #pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k >> 2) * C::kBoxBytes + (k & 3) * 32) >> 4;
                        mma_ss_lo(tmem + w.wg * kBlockN + buf * 32, k_lo + ks * kTileStep + off, q + off,
                                  id, k > 0 ? 1u : 0u);
                    }
                    tc_commit(&sh.st_full[w.wg][buf]);
                }
                __syncwarp();
            }
            continue;
        }
        bool first[2] = {true, true};
        const bool one = !w.pair && nb == 1;
        for (int t = 0; t < 2; ++t) {
            if (t == 1 && one) continue;
            if (!mbar_wait_warp(&sh.q_full[t], q_uses[t] & 1, abort)) goto out;
            ++q_uses[t];
        }
        int prev_v = -1;
        uint32_t prev_use = 0;
        for (int j = 0; j < nb; ++j) {
            const int ks = it % C::kStages, vs = (it + 1) % C::kStages;
            if (!mbar_wait_warp(&sh.kv_full[ks], (it / C::kStages) & 1, abort)) goto out;
            tc_fence_after();
            const uint32_t v_use = (it + 1) / C::kStages;
            it += 2;
            if (w.pair) {
                issue_s(0, ks);
                if (j > 0) {
                    if (!issue_pv(1, prev_v, first[1], false, true)) goto out;
                }
                issue_s(1, ks);
                if (!mbar_wait_warp(&sh.kv_full[vs], v_use & 1, abort)) goto out;
                tc_fence_after();
                if (!issue_pv(0, vs, first[0], j == nb - 1, false)) goto out;
            } else {
                const int t = j & 1;
                issue_s(t, ks);
                if (j > 0) {
                    if (!mbar_wait_warp(&sh.kv_full[prev_v], prev_use & 1, abort)) goto out;
                    tc_fence_after();
                    if (!issue_pv(t ^ 1, prev_v, first[t ^ 1], j == nb - 1, true)) goto out;
                }
            }
            prev_v = vs;
            prev_use = v_use;
        }
        const int t = w.pair ? 1 : (nb - 1) & 1;
        if (one) {
            // of one block the second warpgroup has no tile, but its shares before, and
            // with them their uses of V's slot, are to be over: it says so on its Q
            if (!mbar_wait_warp(&sh.q_full[1], q_uses[1] & 1, abort)) goto out;
            ++q_uses[1];
        }
        if (!w.pair) {
            if (!mbar_wait_warp(&sh.kv_full[prev_v], prev_use & 1, abort)) goto out;
            tc_fence_after();
        }
        if (!issue_pv(t, prev_v, first[t], true, true)) goto out;
    }
out:
    // Wait for every MMA this thread issued before TMEM is released.
    if (elect_one()) tc_commit(&sh.drain[0]);
    __syncwarp();
    mbar_drain_wait(&sh.drain[0], 0);
}

// O^T += V^T P^T of the transposed form: V^T is an MN-major A operand (d
// contiguous), P^T's rows are K-major.  At d = 64 the products' lanes 64-127
// multiply whatever lies behind the V tile and are not read.
template <int D, bool PAGED>
__device__ void mma_issuer_pv(const Params &p, const Table &tab, Shared &sh, uint8_t *sQ, uint8_t *sKV) {
    using C = Cfg<D>;
    volatile int *abort = &sh.abort;
    const uint32_t tmem = sh.tmem_base;
    const uint32_t v_lo = desc_lo(smem_u32(sKV), C::kBoxBytes);
    constexpr uint32_t kTileStep = C::kTileBytes >> 4;
    uint32_t cnt[2] = {0, 0};
    Walker walk;
    walk.begin(p, tab);
    Work w;
    while (walk.next<PAGED>(p, tab, w)) {
        if (!w.few) continue;
        const int nb = w.kb1 - w.kb0, n = few_n(w.it.rows);
        const uint32_t id = idesc_bf16_f32_ab(kBlockM, n, true, false);
        uint32_t it = w.ring + 1;
        for (int j = 0; j < nb; ++j, it += 2) {
            const int vs = it % C::kStages;
            const uint32_t c = cnt[w.wg]++;
            const int b = c & 1;
            // P first: it comes from a warpgroup that has left the shares before,
            // so that V's earlier uses of the slot (of shares skipped above) are over
            if (!mbar_wait_warp(&sh.pt_full[w.wg][b], (c >> 1) & 1, abort)) goto out;
            if (!mbar_wait_warp(&sh.kv_full[vs], (it / C::kStages) & 1, abort)) goto out;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t pt = desc_lo(smem_u32(sQ + w.wg * C::kQBytes + few_p(b)), 16);
                const uint32_t v = v_lo + vs * kTileStep;
                #pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_ss_lo(tmem + C::kColO + w.wg * D, v + ((ks * 2048) >> 4),
                              pt + (((ks >> 2) * n * 128 + (ks & 3) * 32) >> 4), id,
                              (ks > 0 || j > 0) ? 1u : 0u);
                tc_commit(&sh.kv_empty[vs]);
                tc_commit(&sh.pt_empty[w.wg][b]);
            }
            __syncwarp();
        }
    }
out:
    if (elect_one()) tc_commit(&sh.drain[1]);
    __syncwarp();
    mbar_drain_wait(&sh.drain[1], 0);
}

// ---------------------------------------------------------------- softmax
// A thread's running softmax: reference maximum (log2 units) and sum.
struct Row {
    float m, l;
};

// Raises the reference maximum if a row of the warp outgrew it by more than
// the threshold, and rescales O and l with it (P V of the block before is
// done: its completion came with this block's S).
template <int D>
__device__ __forceinline__ void update_max(Row &r, float m_blk, bool first, uint32_t tO) {
    if (first) {
        r.m = m_blk;
        return;
    }
    if (!__any_sync(0xffffffffu, m_blk > r.m + kRescaleThreshold)) return;
    const float m_new = fmaxf(r.m, m_blk);
    const float alpha = (m_new == -INFINITY) ? 1.f : ex2(r.m - m_new);
    #pragma unroll 1
    for (int c = 0; c < D; c += 16) {
        uint32_t ov[16];
        tmem_ld16(tO + c, ov);
        tmem_wait_ld();
        #pragma unroll
        for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
        tmem_st16(tO + c, ov);
    }
    tmem_wait_st();
    r.l *= alpha;
    r.m = m_new;
}

// 64 scores of this thread's row, keys behind `limit` masked.
__device__ __forceinline__ void load_scores(float (&s)[64], uint32_t tS, int col0, int limit) {
    uint32_t raw[64];
    tmem_ld32(tS + col0, raw);
    tmem_ld32(tS + col0 + 32, raw + 32);
    tmem_wait_ld();
    #pragma unroll
    for (int c = 0; c < 64; ++c) s[c] = __uint_as_float(raw[c]);
    if (limit < kBlockN) {
        #pragma unroll
        for (int c = 0; c < 64; ++c)
            if (col0 + c >= limit) s[c] = -INFINITY;
    }
}

// The softmax of one block, by one warp: both halves of its keys, or one (the
// row's other copy has the other).  P_t goes over S_t: keys 0-63 in columns
// 0-31, keys 64-127 in columns 64-95.  Scores are read from tensor memory
// twice, for the maximum and for P: that is cheaper than 128 registers, and a
// loop over the halves keeps the code short.
template <int D>
__device__ __forceinline__ void soft_block(Row &r, int rep, int limit, bool first, float sl2,
                                           uint32_t tS, uint32_t tO, Shared &sh, int t) {
    const int lo = rep == 2 ? (warp_id() & 3) >> 1 : 0, hi = rep == 2 ? lo + 1 : 2;
    float top = -INFINITY;
    #pragma unroll 1
    for (int h = lo; h < hi; ++h) {
        float s[64];
        load_scores(s, tS, h * 64, limit);
        top = fmaxf(top, prefill_impl::row_max64(s));
    }
    update_max<D>(r, top * sl2, first, tO);
    const float mb = r.m == -INFINITY ? 0.f : r.m;
    uint64_t acc = f2pack(0.f, 0.f);
    #pragma unroll 1
    for (int h = lo; h < hi; ++h) {
        float s[64];
        load_scores(s, tS, h * 64, limit);
        uint32_t pk[32];
        prefill_impl::exp_half(s, sl2, mb, pk, acc);
        tmem_st32(tS + h * 64, pk);
        if (rep == 2) {
            #pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = 0u;
            tmem_st32(tS + (1 - h) * 64, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane_id() == 0) {
            if (rep == 2) {
                mbar_arrive(&sh.p_lo[t]);
                mbar_arrive(&sh.p_hi[t]);
            } else {
                mbar_arrive(h ? &sh.p_hi[t] : &sh.p_lo[t]);
            }
        }
    }
    float a0, a1;
    f2unpack(acc, a0, a1);
    r.l += a0 + a1;
}

template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t addr, uint32_t (&r)[N]) {
    if constexpr (N == 4) tmem_ld4(addr, r);
    else if constexpr (N == 8) tmem_ld8(addr, r);
    else if constexpr (N == 16) tmem_ld16(addr, r);
    else tmem_ld32(addr, r);
}
template <int N>
__device__ __forceinline__ void tmem_st_n(uint32_t addr, const uint32_t (&r)[N]) {
    if constexpr (N == 4) tmem_st4(addr, r);
    else if constexpr (N == 8) tmem_st8(addr, r);
    else if constexpr (N == 16) tmem_st16(addr, r);
    else tmem_st32(addr, r);
}

// Sums of N values over a warp; lane l gets that of value l / (32 / N).
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane) {
    #pragma unroll
    for (int m = 16, n = N; m >= 1; m >>= 1) {
        if (n > 1) {
            const bool up = (lane & m) != 0;
            n >>= 1;
            #pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < n) {
                    const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
        }
    }
    return v[0];
}

// What a warpgroup carries from share to share.
struct Count {
    uint32_t s, blocks, o;   // S and P barriers; transposed blocks; O barrier
};

// Q of a share of few rows into buffer b, by asynchronous copies (zeros behind
// the rows), swizzled as TMA would; sent off once they have arrived.
template <int D>
__device__ __forceinline__ void fetch_few_q(const Params &p, const Item &it, int kvh, uint8_t *tile, int b) {
    const int words = (it.rows <= 4 ? 4 : it.rows <= 8 ? 8 : it.rows <= 16 ? 16 : 32) * (D / 8);
    #pragma unroll 1
    for (int x = threadIdx.x & 127; x < words; x += 128) {
        const int row = x / (D / 8), c = x % (D / 8);
        const int at = it.row0 + min(row, it.rows - 1), tok = div_group(p, at);
        const uint16_t *src =
            p.q + ((size_t)(it.tok0 + tok) * p.Hq + kvh * p.G + at - tok * p.G) * D + c * 8;
        copy_async16(tile + few_q(b) + (c >> 3) * Cfg<D>::kBoxBytes + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                     src, row < it.rows);
    }
}
__device__ __forceinline__ void send_few_q(uint64_t *full) {
    copy_async_wait_all();
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(full);
}

// A share of up to RN rows, by one warpgroup: thread = key (of S^T), then
// head-dim index (of O^T).  The reference maxima are the same in all threads.
// False: a wait ran out (in all threads of the warpgroup alike).
template <int D, int RN>
__device__ bool few_rows(const Params &p, const Work &w, Shared &sh, uint8_t *tile, int wg, Count &cnt,
                         float *part_o, float *part_lse) {
    using C = Cfg<D>;
    constexpr int N = RN <= 16 ? 16 : 32;
    const int warp = warp_id(), q4 = warp & 3, lane = lane_id(), tid = threadIdx.x & 127;
    const int bar = 2 + wg;
    const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = sh.tmem_base + lanes + wg * kBlockN;
    const uint32_t tO = sh.tmem_base + lanes + C::kColO + wg * D;
    const int rows = w.it.rows;
    float *red = reinterpret_cast<float *>(&sh.ml[0][0]) + wg * 256;   // [4 warps][32] of this warpgroup
    // (a finite start: no score is below it but -inf, whose P is 0 either way)
    constexpr float kLowest = -3.0e38f;
    float m[RN], l[RN];
    #pragma unroll
    for (int r = 0; r < RN; ++r) {
        m[r] = kLowest;
        l[r] = 0.f;
    }
    const int key = tid;
    uint8_t *pt_key = tile + (key >> 6) * (N * 128) + (key & 7) * 2;
    const int chunk = (key & 63) >> 3;
    bool ok = true;
    for (int j = w.kb0; j < w.kb1; ++j) {
        const uint32_t n = cnt.blocks;
        const int sb = n % kSBufs, pb = n & 1;
        float s[RN];
        bool up = false;
        ok = ok && mbar_wait_warp(&sh.st_full[wg][sb], (n / kSBufs) & 1, &sh.abort);
        if (ok) {
            uint32_t raw[RN];
            tc_fence_after();
            tmem_ld_n<RN>(tS + sb * 32, raw);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.st_empty[wg][sb]);
                if (q4 < 2) mbar_arrive(&sh.kv_empty[(w.ring + 2 * (j - w.kb0)) % C::kStages]);
            }
            const bool seen = w.it.keys - j * kBlockN > key;
            #pragma unroll
            for (int r = 0; r < RN; ++r) {
                s[r] = seen ? __uint_as_float(raw[r]) * p.scale_log2 : -INFINITY;
                up |= s[r] > m[r] + kRescaleThreshold;
            }
        }
        // some key raises a row's maximum by more than the threshold (always in
        // the first block), or a warp has given up
        if (named_bar_or(bar, 128, up || !ok)) {
            if (ok) {
                float top = 0.f;               // lane r: row r's
                #pragma unroll
                for (int r = 0; r < RN; ++r) {
                    const float x = warp_max(s[r]);
                    if (lane == r) top = x;
                }
                if (lane < RN) red[q4 * 32 + lane] = top;
                // P V of the blocks before, which O holds
                if (j > w.kb0) ok = mbar_wait_warp(&sh.pt_empty[wg][pb ^ 1], ((n - 1) >> 1) & 1, &sh.abort);
            }
            if (!named_bar_and(bar, 128, ok)) return false;
            tc_fence_after();
            const int lr = lane & (RN - 1);
            const float top = fmaxf(fmaxf(red[lr], red[32 + lr]), fmaxf(red[64 + lr], red[96 + lr]));
            float alpha[RN];
            #pragma unroll
            for (int r = 0; r < RN; ++r) {
                const float m_new = fmaxf(m[r], __shfl_sync(0xffffffffu, top, r));
                alpha[r] = ex2(m[r] - m_new);
                l[r] *= alpha[r];
                m[r] = m_new;
            }
            if (j > w.kb0) {
                uint32_t ov[RN];
                tmem_ld_n<RN>(tO, ov);
                tmem_wait_ld();
                #pragma unroll
                for (int r = 0; r < RN; ++r) ov[r] = __float_as_uint(__uint_as_float(ov[r]) * alpha[r]);
                tmem_st_n<RN>(tO, ov);
                tmem_wait_st();
            }
        }
        // P^T's buffer of two blocks ago
        ok = mbar_wait_warp(&sh.pt_empty[wg][pb], ((n >> 1) & 1) ^ 1, &sh.abort);
        if (ok) {
            uint8_t *dst = pt_key + few_p(pb);
            #pragma unroll
            for (int r = 0; r < RN; r += 2) {
                const float p0 = ex2(s[r] - m[r]), p1 = ex2(s[r + 1] - m[r + 1]);
                l[r] += p0;
                l[r + 1] += p1;
                const uint32_t pk = pack_bf16(p0, p1);     // off by at most 2^-8 relative
                *reinterpret_cast<uint16_t *>(dst + r * 128 + ((chunk ^ (r & 7)) << 4)) = (uint16_t)pk;
                *reinterpret_cast<uint16_t *>(dst + (r + 1) * 128 + ((chunk ^ ((r + 1) & 7)) << 4)) =
                    (uint16_t)(pk >> 16);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.pt_full[wg][pb]);
        }
        ++cnt.blocks;
    }
    // the last P V: its buffer comes free
    ok = ok && mbar_wait_warp(&sh.pt_empty[wg][(cnt.blocks - 1) & 1], ((cnt.blocks - 1) >> 1) & 1, &sh.abort);
    const float mine = warp_sums<RN>(l, lane);
    if ((lane & (32 / RN - 1)) == 0) red[128 + q4 * 32 + lane / (32 / RN)] = mine;
    if (!named_bar_and(bar, 128, ok)) return false;
    tc_fence_after();
    uint32_t ov[RN];
    tmem_ld_n<RN>(tO, ov);
    tmem_wait_ld();
    const int lr = lane & (RN - 1);            // lane r: row r's sum
    const float sum = (red[128 + lr] + red[160 + lr]) + (red[192 + lr] + red[224 + lr]);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    float *dst = part_o + (size_t)w.slot * D + tid;
    #pragma unroll
    for (int r = 0; r < RN; ++r) {
        const float f = __shfl_sync(0xffffffffu, inv, r);
        if (r < rows && tid < D) dst[r * D] = __uint_as_float(ov[r]) * f;
        if (tid == r && r < rows)
            part_lse[(size_t)w.slot + r] = sum > 0.f ? m[r] + __log2f(sum) : -INFINITY;
    }
    return true;
}

template <int D, bool PAGED>
__device__ void softmax_wg(const Params &p, const Table &tab, Shared &sh, uint8_t *sQ) {
    using C = Cfg<D>;
    const int warp = warp_id(), lane = lane_id(), q4 = warp & 3;
    const int t = warp >> 2;                  // tile of this warpgroup
    const int r = q4 * 32 + lane;             // lane of the tile
    const int kvh = blockIdx.x % p.Hkv;
    const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = sh.tmem_base + lanes + t * kBlockN;
    const uint32_t tO = sh.tmem_base + lanes + C::kColO + t * D;
    float *part_o = p.part_o + (size_t)kvh * p.cap * D;
    float *part_lse = p.part_lse + (size_t)kvh * p.cap;
    Count cnt{0, 0, 0};
    Walker walk;
    walk.begin(p, tab);
    Work w, after;
    // the next share that is this warpgroup's
    auto next = [&](Work &w) -> bool {
        while (walk.next<PAGED>(p, tab, w))
            if (!w.few || w.wg == t) return true;
        return false;
    };
    uint8_t *tile = sQ + t * C::kQBytes;
    uint32_t fewq = 0;
    bool alive = true, have = next(w), fetched = false;
    for (; have; w = after) {
        if (w.few) {
            // Q of the next share is under way while this one is worked on
            if (!fetched) fetch_few_q<D>(p, w.it, kvh, tile, fewq & 1);
            if (alive) send_few_q(&sh.q_full[t]);
            ++fewq;
            have = next(after);
            fetched = have && after.few;
            if (fetched) fetch_few_q<D>(p, after.it, kvh, tile, fewq & 1);
            if (!alive) continue;
            alive = w.it.rows <= 4    ? few_rows<D, 4>(p, w, sh, tile, t, cnt, part_o, part_lse)
                    : w.it.rows <= 8  ? few_rows<D, 8>(p, w, sh, tile, t, cnt, part_o, part_lse)
                    : w.it.rows <= 16 ? few_rows<D, 16>(p, w, sh, tile, t, cnt, part_o, part_lse)
                                      : few_rows<D, 32>(p, w, sh, tile, t, cnt, part_o, part_lse);
            continue;
        }
        have = next(after);
        fetched = false;
        if (!alive) {
            // (this warpgroup gave up: the other one must not wait for it below)
            named_bar_and(1, 256, false);
            break;
        }
        const int step = w.pair ? 1 : 2;
        const int j0 = w.kb0 + (w.pair ? 0 : t);
        const bool used = j0 < w.kb1;
        const int tile0 = w.pair ? t * kBlockM : 0;       // the tile's first row of the item
        const int nrows = min(kBlockM, w.it.rows - tile0);
        const int copy = kBlockM / w.rep;                 // lanes per copy of the rows
        const int lr = r & (copy - 1);                    // this thread's row of the tile
        const bool work = (q4 * 32 & (copy - 1)) < nrows; // some lane of the warp has a row
        bool ok = true;
        if (used) {                                       // Q, swizzled as TMA would write it
            uint4 qv[D / 8];
            const int at = w.it.row0 + tile0 + lr, tok = div_group(p, at);
            const uint4 *src = reinterpret_cast<const uint4 *>(
                p.q + ((size_t)(w.it.tok0 + tok) * p.Hq + kvh * p.G + at - tok * p.G) * D);
            #pragma unroll
            for (int c = 0; c < D / 8; ++c)
                qv[c] = lr < nrows ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
            uint8_t *dst = tile + r * 128;
            #pragma unroll
            for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4 *>(dst + (c >> 3) * C::kBoxBytes + (((c & 7) ^ (r & 7)) << 4)) = qv[c];
            fence_proxy_async_smem();
            tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full[t]);        // (without a tile: this share has begun)
        Row row{-INFINITY, 0.f};
        for (int j = j0; j < w.kb1 && ok; j += step) {
            ok = mbar_wait_warp(&sh.s_full[t], cnt.s & 1, &sh.abort);
            if (!ok) break;
            ++cnt.s;
            tc_fence_after();
            // the block's K slot, handed back by two warps: one of each tile
            // where both read it, else two of this one
            if (lane == 0 && q4 < (w.pair ? 1 : 2))
                mbar_arrive(&sh.kv_empty[(w.ring + 2 * (j - w.kb0)) % C::kStages]);
            if (work) {
                soft_block<D>(row, w.rep, w.it.keys - j * kBlockN, j == j0, p.scale_log2, tS, tO, sh, t);
            } else {
                // no row in these lanes: what P holds there reaches no other lane
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.p_lo[t]);
                    mbar_arrive(&sh.p_hi[t]);
                }
            }
        }
        if (ok && used) {
            ok = mbar_wait_warp(&sh.o_full[t], cnt.o++ & 1, &sh.abort);
            tc_fence_after();
        }
        if (w.pair) {
            // each row has one thread
            if (ok && work) {
                const float inv = row.l > 0.f ? 1.f / row.l : 0.f;
                const size_t at = (size_t)w.slot + tile0 + lr;
                #pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t ov[32];
                    tmem_ld32(tO + c, ov);
                    tmem_wait_ld();
                    if (lr < nrows) {
                        float4 *dst = reinterpret_cast<float4 *>(part_o + at * D + c);
                        #pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e] = make_float4(__uint_as_float(ov[4 * e]) * inv,
                                                 __uint_as_float(ov[4 * e + 1]) * inv,
                                                 __uint_as_float(ov[4 * e + 2]) * inv,
                                                 __uint_as_float(ov[4 * e + 3]) * inv);
                    }
                }
                if (lr < nrows) part_lse[at] = row.l > 0.f ? row.m + __log2f(row.l) : -INFINITY;
            }
            // the warps leave the loop together, or a later barrier would not fill
            if (!named_bar_and(1, 256, ok)) break;
            continue;
        }
        // Both warpgroups, and the copies of the rows, hold parts of the same
        // rows: join them.  Q's tiles are free now (every S is done) and hold
        // the exchange.
        sh.ml[warp][lane] = make_float2(row.m, row.l);
        if (!named_bar_and(1, 256, ok)) break;
        const int quarters = 4 / w.rep;       // warps that hold different rows
        const int mine = q4 & (quarters - 1);
        float M = -INFINITY, L = 0.f;
        float2 part[8];
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
            part[i] = sh.ml[i][lane];
            if ((i & (quarters - 1)) != mine) part[i] = make_float2(-INFINITY, 0.f);
            M = fmaxf(M, part[i].x);
        }
        const float M0 = M == -INFINITY ? 0.f : M;
        #pragma unroll
        for (int i = 0; i < 8; ++i) L = fmaf(part[i].y, ex2(part[i].x - M0), L);
        const float f = row.l > 0.f && L > 0.f ? ex2(row.m - M) / L : 0.f;
        if (t == 0 && q4 < quarters && r < nrows)
            part_lse[(size_t)w.slot + r] = L > 0.f ? M + __log2f(L) : -INFINITY;
        float *buf = reinterpret_cast<float *>(sQ);
        const int warps = w.kb1 - w.kb0 > 1 ? 8 : 4;      // (of one block, the first warpgroup only)
        constexpr int kLd = C::kChunk + 1;
        static_assert(8 * 32 * kLd * 4 <= 2 * C::kQBytes, "exchange within Q's tiles");
        for (int c0 = 0; c0 < D; c0 += C::kChunk) {
            float *dst = buf + (warp * 32 + lane) * kLd;
            if (used && work) {
                uint32_t ov[C::kChunk];
                #pragma unroll
                for (int c = 0; c < C::kChunk; c += 16) tmem_ld16(tO + c0 + c, ov + c);
                tmem_wait_ld();
                #pragma unroll
                for (int e = 0; e < C::kChunk; ++e)
                    dst[e] = f > 0.f ? __uint_as_float(ov[e]) * f : 0.f;
            }
            named_bar_sync(1, 256);
            for (int i = threadIdx.x; i < nrows * C::kChunk; i += 256) {
                const int rr = i / C::kChunk, c = i % C::kChunk;
                float sum = 0.f;
                for (int k = rr >> 5; k < warps; k += quarters) sum += buf[(k * 32 + (rr & 31)) * kLd + c];
                part_o[((size_t)w.slot + rr) * D + c0 + c] = sum;
            }
            named_bar_sync(1, 256);
        }
    }
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
shared_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              const Params p) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *sKV = smem + C::kOffKV;
    Table &tab = *reinterpret_cast<Table *>(smem + C::kOffTable);
    const int warp = warp_id();
    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sh.q_full[t], 4);
            mbar_init(&sh.s_full[t], 1);
            mbar_init(&sh.p_lo[t], 4);
            mbar_init(&sh.p_hi[t], 4);
            mbar_init(&sh.o_full[t], 1);
            mbar_init(&sh.drain[t], 1);
            for (int b = 0; b < kSBufs; ++b) {
                mbar_init(&sh.st_full[t][b], 1);
                mbar_init(&sh.st_empty[t][b], 4);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(&sh.pt_full[t][b], 4);
                mbar_init(&sh.pt_empty[t][b], 1);
            }
        }
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&sh.kv_full[s], 1);
            mbar_init(&sh.kv_empty[s], s & 1 ? 1 : 2);   // V: a commit; K: two softmax warps
        }
        mbar_init(&sh.tail, 1);
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == kWarpMma) tmem_alloc(&sh.tmem_base, kTmemCols);
    if (warp == kWarpK && lane_id() == 0) tma_prefetch_desc(&tmK);
    if (warp == kWarpV && lane_id() == 0) tma_prefetch_desc(&tmV);
    make_plan<PAGED>(p, tab, reinterpret_cast<int *>(smem), sh.scan);
    launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 8) {
        regs_increase<kRegsSoftmax>();
        softmax_wg<D, PAGED>(p, tab, sh, smem);
    } else {
        regs_decrease<kRegsControl>();
        if (warp == kWarpK)
            producer<D, PAGED, false>(&tmK, p, tab, sh, sKV);
        else if (warp == kWarpV)
            producer<D, PAGED, true>(&tmV, p, tab, sh, sKV);
        else if (warp == kWarpMma)
            mma_issuer<D, PAGED>(p, tab, sh, smem, sKV);
        else
            mma_issuer_pv<D, PAGED>(p, tab, sh, smem, sKV);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(sh.tmem_base, kTmemCols);
    }
}

// ---------------------------------------------------------------- combine
// The partials of one (token, query head) row, by SPLIT of a block's eight
// warps: eight where there are few rows and so many partials each, else one.
// Whole calls, 32/8 heads, d = 128, us with eight and one: 32 rows of 32,768
// tokens 33.9 and 37.4, 256 of 4,096 33.4 and 33.8, 384 of 2,048 24.5 and 24.7,
// 448 of 2,048 31.1 and 31.0, 512 34.2 and 33.7 (16/16 heads, d = 64: 54.7 and
// 55.5), 1,024 of 512 21.4 and 19.7, 2,048 of 512 40.1 and 34.6.
constexpr int kCombineWarps = 8;
constexpr int kCombineFewRows = 448;

template <int D, bool PAGED, int SPLIT>
__global__ void __launch_bounds__(32 * kCombineWarps)
shared_combine_kernel(const Params p, uint16_t *__restrict__ o, float *__restrict__ lse,
                      const float *__restrict__ sinks, int tokens) {
    constexpr int PER = D / 32;
    __shared__ float s_acc[SPLIT > 1 ? kCombineWarps : 1][D + 1];
    const int lane = lane_id(), part = warp_id() % SPLIT;
    const long long at = (long long)blockIdx.x * (kCombineWarps / SPLIT) + warp_id() / SPLIT;
    if (at >= (long long)tokens * p.Hq) return;      // (SPLIT = 8: the whole block or none)
    const int tok = (int)(at / p.Hq), h = (int)(at % p.Hq), kvh = h / p.G;
    wait_for_launcher();
    // up to two runs of partials: first row, number, rows apart
    int base[2] = {0, 0}, num[2] = {0, 0}, apart[2] = {0, 0};
    auto take = [&](int k, int item, int row) {
        const int4 t = __ldcg(p.items + item);
        base[k] = t.x + row;
        num[k] = t.y;
        apart[k] = t.z;
    };
    if constexpr (PAGED) {
        const int4 s = __ldcg(p.seqs + tok);
        take(0, s.x, h % p.G);
        if (s.y >= 0) {
            const int row = (tok - s.z) * p.G + h % p.G;
            take(1, s.y + row / kRows, row % kRows);
        }
    } else {
        const int len = p.lens ? __ldg(p.lens + tok / p.Nq) : 0;
        if (len < 0 || len > p.Nk) return;
        const int row = (tok % p.Nq) * p.G + h % p.G;
        take(0, tok / p.Nq * p.pairs + row / kRows, row % kRows);
    }
    const float *po = p.part_o + (size_t)kvh * p.cap * D + lane * PER;
    const float *pl = p.part_lse + (size_t)kvh * p.cap;
    const int n = num[0] + num[1];
    auto row_of = [&](int i) -> size_t {
        return i < num[0] ? (size_t)base[0] + (size_t)i * apart[0]
                          : (size_t)base[1] + (size_t)(i - num[0]) * apart[1];
    };
    const float z = sinks ? __ldg(sinks + h) * 1.4426950408889634f : -INFINITY;
    float m = z;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, __ldcg(pl + row_of(i)));
    #pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float acc[PER], sum = 0.f;
    #pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    if (m != -INFINITY) {
        if (part == 0) sum = ex2(z - m);
        #pragma unroll 4
        for (int i = part; i < n; i += SPLIT) {
            const size_t rr = row_of(i);
            const float wgt = ex2(__ldcg(pl + rr) - m);
            sum += wgt;
            if constexpr (PER == 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(po + rr * D));
                acc[0] = fmaf(wgt, v.x, acc[0]);
                acc[1] = fmaf(wgt, v.y, acc[1]);
                acc[2] = fmaf(wgt, v.z, acc[2]);
                acc[3] = fmaf(wgt, v.w, acc[3]);
            } else {
                const float2 v = __ldcg(reinterpret_cast<const float2 *>(po + rr * D));
                acc[0] = fmaf(wgt, v.x, acc[0]);
                acc[1] = fmaf(wgt, v.y, acc[1]);
            }
        }
    }
    if constexpr (SPLIT > 1) {
        static_assert(SPLIT == kCombineWarps, "one row per block");
        #pragma unroll
        for (int e = 0; e < PER; ++e) s_acc[part][lane * PER + e] = acc[e];
        if (lane == 0) s_acc[part][D] = sum;
        __syncthreads();
        if (part > 0) return;
        #pragma unroll
        for (int k = 1; k < SPLIT; ++k) {
            #pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] += s_acc[k][lane * PER + e];
            sum += s_acc[k][D];
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    uint32_t *dst = reinterpret_cast<uint32_t *>(o + ((size_t)tok * p.Hq + h) * D + lane * PER);
    #pragma unroll
    for (int e = 0; e < PER; e += 2) dst[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    if (lse && lane == 0) {
        const float v = sum > 0.f ? (m + __log2f(sum)) * 0.69314718055994531f : -INFINITY;
        if (PAGED)
            lse[(size_t)tok * p.Hq + h] = v;
        else
            lse[((size_t)(tok / p.Nq) * p.Hq + h) * p.Nq + tok % p.Nq] = v;
    }
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// CTAs per KV head at most; the workspace is sized for them.
int max_shares(int Hkv) { return Hkv >= kSharedMaxCtas ? 1 : kSharedMaxCtas / Hkv; }

// Rows of partials per KV head.  An item gives one per share it touches: all
// rows once, and those of the item at each border between shares once more.
long long part_rows(long long rows, int Hkv, bool twice) {
    return (twice ? 2 : 1) * rows + (long long)max_shares(Hkv) * (rows < kRows ? rows : kRows);
}

struct Workspace {
    size_t o, lse, items, seqs, bytes;
};

Workspace layout(long long rows, int Hkv, int d, bool paged) {
    const size_t n = (size_t)part_rows(rows, Hkv, paged) * Hkv;
    Workspace w;
    w.o = 0;
    w.lse = up256(n * d * sizeof(float));
    w.items = w.lse + up256(n * sizeof(float));
    w.seqs = w.items + kMaxItems * sizeof(int4);
    w.bytes = w.seqs + kMaxSeqs * sizeof(int4);
    return w;
}

template <int D, bool PAGED>
int launch(const CUtensorMap &tk, const CUtensorMap &tv, const Params &p, const SharedArgs &a,
           cudaStream_t stream) {
    using C = Cfg<D>;
    constexpr int smem = C::kOffTable + (int)sizeof(Table) + 1024;
    static_assert(smem + sizeof(Shared) <= 232448, "shared memory");
    // (on every call: the attribute goes with the device's context)
    if (cudaFuncSetAttribute(shared_kernel<D, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem) != cudaSuccess)
        return -5;
    shared_kernel<D, PAGED><<<p.n * p.Hkv, kThreads, smem, stream>>>(tk, tv, p);
    if (cudaGetLastError() != cudaSuccess) return -5;
    // The combine is set up while the main kernel's last CTAs run.
    const int tokens = p.S * p.Nq;
    const long long rows = (long long)tokens * p.Hq;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    const bool few = rows <= kCombineFewRows;
    const int per = few ? 1 : kCombineWarps;
    cfg.gridDim = dim3((unsigned)((rows + per - 1) / per));
    cfg.blockDim = dim3(32 * kCombineWarps);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, few ? shared_combine_kernel<D, PAGED, kCombineWarps>
                                        : shared_combine_kernel<D, PAGED, 1>,
                              p, static_cast<uint16_t *>(a.o), a.lse, a.sinks, tokens) == cudaSuccess
               ? 0 : -5;
}

int launch_any(const SharedArgs &a, cudaStream_t stream) {
    if (a.S <= 0 || a.Nq <= 0) return 0;
    const int G = a.Hq / a.Hkv;
    const long long rows = (long long)a.S * a.Nq * G;
    const Workspace ws = layout(rows, a.Hkv, a.d, a.paged);
    if (!a.workspace || a.workspace_bytes < ws.bytes) return -4;
    Params p{};
    p.q = static_cast<const uint16_t *>(a.q);
    p.block_table = a.block_table;
    p.lens = a.lens;
    p.cu_groups = a.cu_groups;
    p.prefix_lens = a.prefix_lens;
    char *base = static_cast<char *>(a.workspace);
    p.part_o = reinterpret_cast<float *>(base + ws.o);
    p.part_lse = reinterpret_cast<float *>(base + ws.lse);
    p.items = reinterpret_cast<int4 *>(base + ws.items);
    p.seqs = reinterpret_cast<int4 *>(base + ws.seqs);
    p.S = a.S;
    p.num_groups = a.num_groups;
    p.num_pages = a.num_pages;
    p.max_pages = a.max_pages;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = G;
    p.G_magic = G > 1 ? (uint32_t)(((1ull << 32) + G - 1) / G) : 0u;
    p.Nq = a.Nq;
    p.Nk = a.Nk;
    p.pairs = (a.Nq * G + kRows - 1) / kRows;
    const int sms = device_sm_count() < kSharedMaxCtas ? device_sm_count() : kSharedMaxCtas;
    p.n = a.Hkv >= sms ? 1 : sms / a.Hkv;
    p.total_k = a.paged ? 0 : a.S_all * a.Nk;
    p.cap = part_rows(rows, a.Hkv, a.paged);
    p.cost_few = a.d == 128 ? Cost<128>::kFew : Cost<64>::kFew;
    p.cost_one = a.d == 128 ? Cost<128>::kOne : Cost<64>::kOne;
    p.cost_pair = a.d == 128 ? Cost<128>::kPair : Cost<64>::kPair;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    // K/V rows: the cache's slots, read a page box at a time, or the sequences' stored keys
    alignas(64) CUtensorMap tk, tv;
    const bool none = !a.paged && p.total_k == 0;   // no key at all: the maps are not used
    const void *k = none ? a.q : a.k, *v = none ? a.q : a.v;
    const uint64_t TK = none ? 1 : a.paged ? (uint64_t)a.num_pages * kPage : (uint64_t)p.total_k;
    const uint64_t s1 = (uint64_t)a.d * 2, s2 = (uint64_t)a.Hkv * a.d * 2;
    const uint32_t box = a.paged ? kPage : kBlockN;
    if (encode_tensor_map_3d(&tk, k, 2, a.d, a.Hkv, TK, s1, s2, 64, 1, box, 128) ||
        encode_tensor_map_3d(&tv, v, 2, a.d, a.Hkv, TK, s1, s2, 64, 1, box, 128))
        return -5;
    if (a.d == 128)
        return a.paged ? launch<128, true>(tk, tv, p, a, stream) : launch<128, false>(tk, tv, p, a, stream);
    if (a.d == 64)
        return a.paged ? launch<64, true>(tk, tv, p, a, stream) : launch<64, false>(tk, tv, p, a, stream);
    return -2;
}

}  // namespace shared_impl

size_t shared_workspace_bytes(long long rows_per_kvh, int Hkv, int d, bool paged) {
    return shared_impl::layout(rows_per_kvh, Hkv, d, paged).bytes;
}

int launch_shared(const SharedArgs &a, cudaStream_t stream) {
    return shared_impl::launch_any(a, stream);
}

}  // namespace fa
