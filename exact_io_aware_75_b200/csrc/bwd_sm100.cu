// bwd_sm100.cu -- exact attention backward (dQ, dK, dV) on the sm_100a tensor
// core.
//
// What it computes: for O = softmax(Q K^T * scale + mask) V and an upstream
// gradient dO, the gradients of sum(dO * O) with respect to Q, K and V.  The
// attention matrix is never stored: it is recomputed from Q, K and the row
// log-sum-exp the forward saved ("FlashAttention: same math, different IO" in
// samanvya.dev's "Attention Is the Bottleneck": the backward rebuilds the
// matrix instead of keeping it, trading FLOPs for memory traffic).  With
// D_i = dO_i . O_i, for each visible (query i, key j):
//     P_ij  = 2^(S_ij * scale * log2e - LSE_i * log2e)
//     dS_ij = P_ij (dO_i . V_j - D_i)
//     dV_j += P_ij dO_i,   dK_j += scale dS_ij Q_i,   dQ_i += scale dS_ij K_j
// and grouped query heads add into their shared KV head's dK, dV.
//
// How (B200 design):
//   * bwd_prep_kernel: D = rowsum(O * dO) per (token, head), and zeroes the
//     fp32 dQ accumulator.
//   * bwd_kernel, persistent, one CTA per SM.  A work unit is one KV head's
//     block of 128 keys; K_j and V_j stay in shared memory while the unit walks
//     every (query head of the group, 64-row query tile) that sees the block.
//     dK_j and dV_j accumulate in tensor memory for the whole unit, so the GQA
//     sum over query heads costs nothing and each unit writes its rows once.
//   * Per tile, five tcgen05 GEMMs, all with the 128 keys on the TMEM lanes:
//       S^T  = K_j Q_t^T        (128 x 64, K = d)
//       dP^T = V_j dO_t^T       (128 x 64, K = d)
//       dV  += P^T dO_t         (128 x d,  K = 64; P^T read from TMEM)
//       dK  += dS^T Q_t         (128 x d,  K = 64; dS^T from shared memory)
//       dQ^T = K_j^T dS^T       (d x 64,   K = 128; lands on dP^T's columns)
//     S^T and dP^T are double-buffered in TMEM (2 x 2 x 64 columns) and dK, dV
//     take 2 x 128: the 512 columns of the SM.  Two softmax warpgroups take
//     alternate tiles, so one tile's elementwise work overlaps the next tile's
//     GEMMs.
//   * Warps 8-11 drain dQ^T from TMEM, stage it transposed in shared memory
//     and add it into the fp32 accumulator with TMA reduce-adds (the adds
//     happen in L2, 16 KB per operation); bwd_convert_kernel rounds the
//     accumulator to bf16 at the end.
//   * Warp 12 loads K_j, V_j once per unit and Q_t, dO_t per tile by TMA into
//     a 3-slot ring (6 at d = 64), with the tile's LSE (in log2 units) and D beside them.
//     Two threads issue the MMAs: warp 13 S^T and dP^T (and owns the TMEM
//     allocation), warp 14 the three gradient GEMMs, so that a tile's S^T
//     never waits behind the previous tile's gradients (which wait for that
//     tile's softmax) and the two issue streams overlap.
#include <type_traits>
#include <cuda.h>
#include <cuda_runtime.h>

#include "balance.cuh"
#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {

namespace bwd_impl {

// Widest head dim.  d = 64 takes one 64-column box of each tile instead of two
// (and half the products' steps or columns); only dQ^T keeps M = 128, whose
// lanes 64-127 multiply what lies behind the K box and are not read.  Against
// zero-padded 128-wide tiles: 380 us for 428 (packed cross attention, 24 pairs
// of up to 1,024 x 2,048, 16 heads); with the longer ring and the second set of
// K and V below 343.  d = 64 also has the tensor memory for a third tile in
// flight, or for a second set of dV and dK to let a unit's last rows be written
// behind the next one's first tile: 359 and 377, so neither is done.  What
// bounds a tile is its way through the five products and the elementwise pass
// between them: of 4,700 cycles for a warpgroup's tile the pass takes 1,930,
// the wait for the next S^T the rest.
constexpr int kD = 128;
constexpr int kBlockK = 128;   // keys per unit
constexpr int kBlockQ = 64;    // queries per tile
constexpr int kPartQ = 16;     // queries per step of the elementwise pass
constexpr int kThreads = 512;
constexpr int kWarpDrain = 8;  // warps 8..11
constexpr int kWarpTma = 12;
constexpr int kWarpMma = 13;       // S^T, dP^T; TMEM allocation
constexpr int kWarpMmaGrad = 14;   // dV, dK, dQ^T
// Slots of the Q/dO ring.  A slot is free again when its tile's dK is done, so
// with three the next load starts little more than a tile's time before it is
// needed: about the latency of HBM.  d = 64 has room for six (367 us for 375
// with one set of K and V, below).
template <int DH>
constexpr int kStages = DH == 64 ? 6 : 3;
// Register split (launched with 512 x 128 = 65,536): the two elementwise
// warpgroups hold two 16-column steps of Sᵀ and dPᵀ at a time (one being
// computed, the next in flight from TMEM).
constexpr int kRegsSoftmax = 176;
constexpr int kRegsDrain = 88;
constexpr int kRegsControl = 72;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsDrain + 128 * kRegsControl <= kThreads * 128,
              "register split");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;     // S^T of buffer b at b * 64 (P^T overwrites its first 32)
constexpr uint32_t kColDP = 128;  // dP^T of buffer b at 128 + b * 64, then the tile's dQ^T
constexpr uint32_t kColDV = 256;
constexpr uint32_t kColDK = 384;

// Sets of K and V tiles.  At d = 64 half of each tile's place is unused
// otherwise: a unit's K and V are loaded while the unit before it finishes.
template <int DH>
constexpr int kSets = DH == 64 ? 2 : 1;

constexpr int kKVBox = kBlockK * 64 * 2;         // 128 rows x 64 bf16 (16 KB)
constexpr int kKVTile = kBlockK * kD * 2;        // 32 KB
constexpr int kQBox = kBlockQ * 64 * 2;          // 64 rows x 64 bf16 (8 KB)
constexpr int kQTile = kBlockQ * kD * 2;         // 16 KB
constexpr int kDSBytes = kBlockK * kBlockQ * 2;  // 16 KB
constexpr int kOffK = 0;
constexpr int kOffV = kKVTile;
constexpr int kOffStage = 2 * kKVTile;           // stage s: Q_t then dO_t
template <int DH>
constexpr int kStageBytes = 2 * kBlockQ * DH * 2;
constexpr int kOffDS = kOffStage + 3 * 2 * kQTile;
static_assert(kStages<64> * kStageBytes<64> == kOffDS - kOffStage &&
              kStages<128> * kStageBytes<128> == kOffDS - kOffStage, "Q/dO ring");
constexpr int kDQHalf = 32;                      // dQ rows per reduce-add
constexpr int kDQBytes = kDQHalf * kD * 4;       // 16 KB staging buffer
constexpr int kOffDQ = kOffDS + 2 * kDSBytes;    // two staging buffers
// stage s: lse2[64], D[64] (fp32); d = 64 leaves half of a staging buffer unused
constexpr int kRowBytes = 2 * kBlockQ * 4;
template <int DH>
constexpr int kOffRows = DH == 64 ? kOffDQ + kDQHalf * DH * 4 : kOffDQ + 2 * kDQBytes;
static_assert(kDQHalf * 64 * 4 + kStages<64> * kRowBytes <= kDQBytes, "rows of the ring");
constexpr int kSmemBytes = kOffRows<128> + kStages<128> * kRowBytes + 1024;
constexpr int kBarDrain = 1;                     // named barrier of the dQ warps

struct Params {
    const float *lse;   // saved row log-sum-exp (natural log)
    const float *dd;    // D = rowsum(O * dO), same layout as lse
    float *dq_acc;      // [total, Hq, d] fp32
    void *dk, *dv;      // [total, Hkv, d] bf16
    const int *cu_seqlens;
    int num_seqs, seqlen, total_tokens, max_seqlen;
    int Hq, Hkv, group;
    int causal, window;
    float scale, scale_log2;
    int num_kblocks, num_units;
    // Cross attention: keys and values are tensors of their own, dense
    // [num_seqs, seqlen_k] of which seq_lens_k[s] (if given) are visible, or
    // packed by cu_seqlens_k.
    const int *cu_seqlens_k, *seq_lens_k;
    int seqlen_k, total_k, max_seqlen_k;
};

struct Unit {
    int seq, kvh, tok0, L;
    int j0, jl;        // first and last key of the block (local to the sequence)
    int t_lo, nt;      // query tiles [t_lo, t_lo + nt) of each query head
    int ntiles;        // group * nt
    int tokk0, Lk;     // first key and visible keys (tok0 and L but for cross attention)
    // cross attention: stored keys; those past Lk get zero gradients, from the
    // head's last unit
    int Ls;
    bool last;
};

// Cross attention: where a sequence's queries and keys lie (Ls: its stored
// keys, of which Lk are visible); false if they do not fit.
__device__ __forceinline__ bool cross_lengths(const Params &p, int s, int &tok0, int &L, int &tokk0,
                                              int &Lk, int &Ls) {
    if (p.cu_seqlens) {
        tok0 = __ldg(p.cu_seqlens + s);
        L = __ldg(p.cu_seqlens + s + 1) - tok0;
        tokk0 = __ldg(p.cu_seqlens_k + s);
        Ls = Lk = __ldg(p.cu_seqlens_k + s + 1) - tokk0;
        return tok0 >= 0 && L >= 0 && L <= p.max_seqlen && tok0 <= p.total_tokens - L && tokk0 >= 0 &&
               Lk >= 0 && Lk <= p.max_seqlen_k && tokk0 <= p.total_k - Lk;
    }
    tok0 = s * p.seqlen;
    L = p.seqlen;
    tokk0 = s * p.seqlen_k;
    Ls = p.seqlen_k;
    Lk = p.seq_lens_k ? __ldg(p.seq_lens_k + s) : p.seqlen_k;
    return Lk >= 0 && Lk <= p.seqlen_k;
}

// A sequence's units, by their query tiles.  The last unit also clears the
// gradients of keys that no query sees; a sequence without any (query, key)
// pair has one unit for that.
struct CrossUnits {
    const Params &p;
    __device__ __forceinline__ SeqUnits operator()(int s) const {
        int tok0, L, tokk0, Lk, Ls;
        if (!cross_lengths(p, s, tok0, L, tokk0, Lk, Ls)) {
            report_error(kDevErrInput);
            return SeqUnits{0, 0};
        }
        if (Ls == 0) return SeqUnits{0, 0};
        if (L == 0 || Lk == 0) return SeqUnits{1, 0};
        return SeqUnits{(Lk + kBlockK - 1) / kBlockK, (L + kBlockQ - 1) / kBlockQ};
    }
};

// False if the unit has no (query, key) pair.
template <bool CROSS, class U>
__device__ __forceinline__ bool get_unit(const U &u_, const Params &p, Unit &w) {
    if constexpr (CROSS) {
        w.seq = u_.s;
        w.kvh = u_.h;
        w.j0 = u_.k * kBlockK;
        w.last = false;
        if (!cross_lengths(p, w.seq, w.tok0, w.L, w.tokk0, w.Lk, w.Ls)) {
            report_error(kDevErrInput);
            return false;
        }
        if (w.L == 0 || w.Lk == 0) {
            w.last = u_.k == 0;
            return false;
        }
        if (w.j0 >= w.Lk) return false;
        w.last = w.j0 + kBlockK >= w.Lk;
        w.jl = min(w.Lk, w.j0 + kBlockK) - 1;
        w.t_lo = 0;
        w.nt = (w.L + kBlockQ - 1) / kBlockQ;
        w.ntiles = p.group * w.nt;
        return true;
    } else {
    const int u = u_;
    const int per = p.num_seqs * p.Hkv;
    const int jb = u / per;           // causal: low key blocks are the heaviest
    const int r = u % per;
    w.seq = r / p.Hkv;
    w.kvh = r % p.Hkv;
    if (p.cu_seqlens) {
        w.tok0 = __ldg(p.cu_seqlens + w.seq);
        w.L = __ldg(p.cu_seqlens + w.seq + 1) - w.tok0;
        // A sequence outside [0, total_tokens) or longer than max_seqlen is
        // skipped by every role alike and reported.
        if (w.tok0 < 0 || w.L < 0 || w.L > p.max_seqlen || w.tok0 > p.total_tokens - w.L) {
            report_error(kDevErrInput);
            return false;
        }
    } else {
        w.tok0 = w.seq * p.seqlen;
        w.L = p.seqlen;
    }
    w.j0 = jb * kBlockK;
    w.tokk0 = w.tok0;
    w.Lk = w.L;
    if (w.L <= 0 || w.j0 >= w.Lk) return false;
    w.jl = min(w.Lk, w.j0 + kBlockK) - 1;
    const int nq = (w.L + kBlockQ - 1) / kBlockQ;
    int lo = 0, hi = nq;
    if (p.causal) {
        lo = w.j0 / kBlockQ;                        // queries i >= j0
        if (p.window > 0) hi = min(nq, (w.jl + p.window - 1) / kBlockQ + 1);  // i < jl + W
    }
    w.t_lo = lo;
    w.nt = hi - lo;
    w.ntiles = p.group * w.nt;
    return w.nt > 0;
    }
}

__device__ __forceinline__ void tile_of(const Unit &w, const Params &p, int k, int &h, int &q0) {
    h = w.kvh * p.group + k / w.nt;
    q0 = (w.t_lo + k % w.nt) * kBlockQ;
}

__device__ __forceinline__ size_t row_index(const Params &p, const Unit &w, int h, int i) {
    return p.cu_seqlens ? (size_t)h * p.total_tokens + w.tok0 + i
                        : ((size_t)w.seq * p.Hq + h) * p.seqlen + i;
}

__device__ __forceinline__ int sched_unit(int it) {
    const int G = gridDim.x, b = blockIdx.x;
    return (it & 1) ? (it + 1) * G - 1 - b : it * G + b;
}

struct UnitIndex {
    int it = 0, u = 0;
    __device__ __forceinline__ operator int() const { return u; }
};
// (or cross attention's order of the units, balance.cuh)
template <bool CROSS, class S, class W>
__device__ __forceinline__ bool unit_more(const Params &p, const S &sh, W &w) {
    if constexpr (CROSS) {
        return w.more(*sh.deal, p.num_seqs, p.Hkv, p.num_kblocks);
    } else {
        for (; w.it * (int)gridDim.x < p.num_units; ++w.it)
            if ((w.u = sched_unit(w.it)) < p.num_units) return true;
        return false;
    }
}
#define FOR_EACH_BWD_UNIT(u)                                                               \
    for (std::conditional_t<CROSS, DealWalk, UnitIndex> u; unit_more<CROSS>(p, sh, u); ++u.it)

struct Shared {
    uint64_t kv_full[2], kv_empty[2];        // by set
    uint64_t qd_full[kStages<64>], qd_empty[kStages<64>];
    uint64_t s_full[2], p_full[2], dq_full[2], dq_free[2];
    uint64_t pt_free[2];     // dV of the buffer's tile done: Sᵀ's columns are free
    uint64_t ds_free[2];     // dK of the buffer's tile done: its dSᵀ buffer is free
    uint64_t acc_full, acc_free;
    uint64_t drain[2];
    // cross attention: bytes of tiles with rows to clear; the order of the units
    uint64_t kv_tail, qd_tail;
    DealTable *deal;
    uint32_t tmem_base;
    int abort;
};
static_assert(kSmemBytes + sizeof(Shared) <= 232448, "shared memory");

// Cross attention: zeros over rows [valid, rows) of a tile of 64-column
// boxes, one warp.  What lies behind a sequence's end (other sequences,
// padding, NaN included) would otherwise meet P = 0 or dS = 0 in a product.
template <int DH>
__device__ __forceinline__ void clear_rows(uint8_t *tile, int rows, int valid, int box_bytes) {
    const int n16 = (rows - valid) * 8;
    for (int b = 0; b < DH / 64; ++b)
        for (int i = lane_id(); i < n16; i += 32)
            *reinterpret_cast<uint4 *>(tile + b * box_bytes + valid * 128 + i * 16) =
                make_uint4(0u, 0u, 0u, 0u);
}

// ------------------------------------------------------------- TMA producer
template <int DH, bool CROSS>
__device__ void producer(const CUtensorMap *tmQ, const CUtensorMap *tmK, const CUtensorMap *tmV,
                         const CUtensorMap *tmdO, const Params &p, Shared &sh, uint8_t *smem) {
    volatile int *abort = &sh.abort;
    const int lane = lane_id();
    float *rows = reinterpret_cast<float *>(smem + kOffRows<DH>);
    uint32_t uc = 0, n = 0, kv_tails = 0, qd_tails = 0;
    FOR_EACH_BWD_UNIT(u) {
        Unit w;
        if (!get_unit<CROSS>(u, p, w)) continue;
        // LSE and D of a tile's rows, asked for a tile ahead: with their latency in
        // each step this warp set the ring's pace (S^T waited 500 cycles a tile for
        // Q and dO at d = 64, 1,100 at 128; now 110 and 710).  8 x 2,048, 16
        // heads, d = 64: 760 to 600 us, causal 430 to 348; 4,096, 32/8 heads,
        // d = 128: 747 to 718 with the two small kernels, causal 391 to 384.
        float next_l[2], next_d[2];
        auto ask_rows = [&](int k) {
            int h, q0;
            tile_of(w, p, k, h, q0);
            #pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = q0 + lane + 32 * e;
                next_l[e] = INFINITY;
                next_d[e] = 0.f;
                if (i < w.L) {
                    const size_t idx = row_index(p, w, h, i);
                    next_l[e] = __ldg(p.lse + idx);
                    next_d[e] = __ldg(p.dd + idx);
                }
            }
        };
        ask_rows(0);
        const int set = uc % kSets<DH>;
        uint8_t *tK = smem + kOffK + set * kKVBox, *tV = smem + kOffV + set * kKVBox;
        if (!mbar_wait_warp(&sh.kv_empty[set], ((uc / kSets<DH>) & 1) ^ 1, abort)) goto out;
        const bool kv_clear = CROSS && w.Lk - w.j0 < kBlockK && w.tokk0 + w.Lk < p.total_k;
        uint64_t *kv_bar = kv_clear ? &sh.kv_tail : &sh.kv_full[set];
        if (lane == 0) {
            mbar_arrive_expect_tx(kv_bar, 2 * kBlockK * DH * 2);
            for (int b = 0; b < DH / 64; ++b) {
                tma_load_3d(tK + b * kKVBox, tmK, kv_bar, b * 64, w.kvh, w.tokk0 + w.j0);
                tma_load_3d(tV + b * kKVBox, tmV, kv_bar, b * 64, w.kvh, w.tokk0 + w.j0);
            }
        }
        ++uc;
        if (kv_clear) {
            ++kv_tails;
            if (!mbar_wait_warp(&sh.kv_tail, (kv_tails - 1) & 1, abort)) goto out;
            clear_rows<DH>(tK, kBlockK, w.Lk - w.j0, kKVBox);
            clear_rows<DH>(tV, kBlockK, w.Lk - w.j0, kKVBox);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.kv_full[set]);
        }
        // A head's last tile may hold rows to clear.  It has a step of its own behind
        // the loop over the others: with the wait and the loops for it in every tile's
        // way the loads asked for ahead were waited for there, and cross attention was
        // slower than without asking ahead.  Cross, 16 heads, d = 64, us without asking
        // / asking with one loop / so: 37 x 512 queries on 2,048 keys 845 / 891 / 853,
        // 37 x 1,024 on 512 448 / 417 / 388, 9 x 2,048 on 2,048 695 / 766 / 696; 32/8
        // heads 1,357 / 1,435 / 1,279.  d = 128, 32/8 heads, 9 x 2,048 on 2,048 1,710 /
        // 1,649 / 1,662.
        const bool q_clear = CROSS && w.L % kBlockQ != 0 && w.tok0 + w.L < p.total_tokens;
        auto step = [&](int k, auto clear) -> bool {
            const int s = n % kStages<DH>;
            if (!mbar_wait_warp(&sh.qd_empty[s], ((n / kStages<DH>) & 1) ^ 1, abort)) return false;
            int h, q0;
            tile_of(w, p, k, h, q0);
            uint8_t *st = smem + kOffStage + s * kStageBytes<DH>;
            uint64_t *bar = clear ? &sh.qd_tail : &sh.qd_full[s];
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, 2 * kBlockQ * DH * 2);
                for (int b = 0; b < DH / 64; ++b) {
                    tma_load_3d(st + b * kQBox, tmQ, bar, b * 64, h, w.tok0 + q0);
                    tma_load_3d(st + kBlockQ * DH * 2 + b * kQBox, tmdO, bar, b * 64, h, w.tok0 + q0);
                }
            }
            // The tile's -LSE (log2 units) and -D; rows past the sequence get
            // LSE = +inf, so their P is exactly 0.
            float *rs = rows + s * 2 * kBlockQ;
            const float l[2] = {next_l[0], next_l[1]}, dv[2] = {next_d[0], next_d[1]};
            if (k + 1 < w.ntiles) ask_rows(k + 1);
            #pragma unroll
            for (int e = 0; e < 2; ++e) {
                rs[lane + 32 * e] = -(l[e] * 1.4426950408889634f);
                rs[kBlockQ + lane + 32 * e] = -dv[e];
            }
            if (clear) {
                ++qd_tails;
                if (!mbar_wait_warp(&sh.qd_tail, (qd_tails - 1) & 1, abort)) return false;
                clear_rows<DH>(st, kBlockQ, w.L - q0, kQBox);
                clear_rows<DH>(st + kBlockQ * DH * 2, kBlockQ, w.L - q0, kQBox);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.qd_full[s]);
                if (clear) mbar_arrive(&sh.qd_full[s]);   // in place of the byte count
            }
            return true;
        };
        const int plain = w.nt - (q_clear ? 1 : 0);
        for (int k = 0; k < w.ntiles;) {
            for (const int end = k + plain; k < end; ++k, ++n)
                if (!step(k, std::false_type{})) goto out;
            if (q_clear) {
                if (!step(k, std::true_type{})) goto out;
                ++k;
                ++n;
            }
        }
    }
    return;
out:
    if (lane == 0) {
        if (kv_tails) mbar_drain_wait(&sh.kv_tail, (kv_tails - 1) & 1);
        if (qd_tails) mbar_drain_wait(&sh.qd_tail, (qd_tails - 1) & 1);
        for (int i = 0; i < kSets<DH>; ++i)
            if (uc > (uint32_t)i) mbar_drain_wait(&sh.kv_full[i], ((uc - 1 - i) / kSets<DH>) & 1);
        for (int s = 0; s < kStages<DH>; ++s)
            if (n > (uint32_t)s) mbar_drain_wait(&sh.qd_full[s], ((n - 1 - s) / kStages<DH>) & 1);
    }
}

// ----------------------------------------------------------- MMA issuers
// S^T(b) = K Q^T and dP^T(b) = V dO^T: K-major operands, d/16 steps; a step
// moves 32 bytes inside a 64-column box, 4 steps cross to the next box.  S^T
// of tile n overwrites the P^T that dV of tile n-2 reads, so it waits for
// that MMA to complete; dP^T overwrites the dQ^T of tile n-2, so it waits
// until that is drained.
template <int DH, bool CROSS>
__device__ void mma_issuer_s(const Params &p, Shared &sh, uint8_t *smem) {
    volatile int *abort = &sh.abort;
    const uint32_t tmem = sh.tmem_base;
    const uint32_t idS = idesc_bf16_f32_ab(kBlockK, kBlockQ, false, false);
    const uint32_t aStage = smem_u32(smem + kOffStage);
    uint32_t uc = 0, n = 0;
    FOR_EACH_BWD_UNIT(u) {
        Unit w;
        if (!get_unit<CROSS>(u, p, w)) continue;
        const int set = uc % kSets<DH>;
        const uint32_t kLo = desc_lo(smem_u32(smem + kOffK + set * kKVBox), 16);
        const uint32_t vLo = desc_lo(smem_u32(smem + kOffV + set * kKVBox), 16);
        if (!mbar_wait(&sh.kv_full[set], (uc / kSets<DH>) & 1, abort)) goto out;
        ++uc;
        for (int k = 0; k < w.ntiles; ++k, ++n) {
            const int b = n & 1, s = n % kStages<DH>;
            if (!mbar_wait(&sh.qd_full[s], (n / kStages<DH>) & 1, abort)) goto out;
            if (n >= 2 && !mbar_wait(&sh.pt_free[b], ((n - 2) >> 1) & 1, abort)) goto out;
            tc_fence_after();
            const uint32_t qLo = desc_lo(aStage + s * kStageBytes<DH>, 16);
            const uint32_t dLo = qLo + (kBlockQ * DH * 2 >> 4);
            #pragma unroll
            for (int ks = 0; ks < DH / 16; ++ks) {
                const uint32_t okv = ((ks >> 2) * kKVBox + (ks & 3) * 32) >> 4;
                const uint32_t oq = ((ks >> 2) * kQBox + (ks & 3) * 32) >> 4;
                mma_ss_lo(tmem + kColS + b * kBlockQ, kLo + okv, qLo + oq, idS, ks > 0);
            }
            if (n >= 2 && !mbar_wait(&sh.dq_free[b], ((n - 2) >> 1) & 1, abort)) goto out;
            tc_fence_after();
            #pragma unroll
            for (int ks = 0; ks < DH / 16; ++ks) {
                const uint32_t okv = ((ks >> 2) * kKVBox + (ks & 3) * 32) >> 4;
                const uint32_t oq = ((ks >> 2) * kQBox + (ks & 3) * 32) >> 4;
                mma_ss_lo(tmem + kColDP + b * kBlockQ, vLo + okv, dLo + oq, idS, ks > 0);
            }
            tc_commit(&sh.s_full[b]);
        }
        tc_commit(&sh.kv_empty[set]); // K_j, V_j read by this thread's MMAs
    }
out:
    tc_commit(&sh.drain[0]);
    mbar_drain_wait(&sh.drain[0], 0);
}

// dQ^T = K^T dS^T (K = 128 keys), then dV += P^T dO and dK += dS^T Q (K = 64
// queries), once the tile's softmax has published P^T (TMEM) and dS^T (shared
// memory).  dQ^T goes first so its drain, which the next dP^T on these
// columns waits for, starts early; each step is committed on its own
// barrier: dQ^T (drain may read), dV (S^T's columns free), dK (dS^T and the
// Q/dO slot free).  dO and Q are MN-major B operands (d contiguous; 16 query rows
// per step, boxes of 64 columns LBO apart); dS^T sits in shared memory as 128
// key rows of 64 queries, 128-byte swizzled: K-major A for dK, MN-major B
// for dQ^T.
template <int DH, bool CROSS>
__device__ void mma_issuer_grad(const Params &p, Shared &sh, uint8_t *smem) {
    volatile int *abort = &sh.abort;
    const uint32_t tmem = sh.tmem_base;
    const uint32_t idAcc = idesc_bf16_f32_ab(kBlockK, DH, false, true);
    const uint32_t idDQ = idesc_bf16_f32_ab(kD, kBlockQ, true, true);
    const uint32_t aStage = smem_u32(smem + kOffStage), aDS = smem_u32(smem + kOffDS);
    uint32_t uc = 0, m = 0;
    FOR_EACH_BWD_UNIT(u) {
        Unit w;
        if (!get_unit<CROSS>(u, p, w)) continue;
        const int set = uc % kSets<DH>;
        const uint32_t kLoMN = desc_lo(smem_u32(smem + kOffK + set * kKVBox), kKVBox);
        if (!mbar_wait(&sh.kv_full[set], (uc / kSets<DH>) & 1, abort)) goto out;
        ++uc;
        for (int k = 0; k < w.ntiles; ++k, ++m) {
            const bool first = k == 0;
            const int b = m & 1, s = m % kStages<DH>;
            if (!mbar_wait(&sh.p_full[b], (m >> 1) & 1, abort)) goto out;
            if (first && uc > 1 && !mbar_wait(&sh.acc_free, (uc - 2) & 1, abort)) goto out;
            tc_fence_after();
            const uint32_t q = aStage + s * kStageBytes<DH>, dO = q + kBlockQ * DH * 2;
            const uint32_t ds = aDS + b * kDSBytes;
            const uint32_t qLoMN = desc_lo(q, kQBox), dLoMN = desc_lo(dO, kQBox);
            const uint32_t dsLoK = desc_lo(ds, 16), dsLoMN = desc_lo(ds, kDSBytes);
            #pragma unroll
            for (int ks = 0; ks < kBlockK / 16; ++ks)
                mma_ss_lo(tmem + kColDP + b * kBlockQ, kLoMN + ((ks * 2048) >> 4),
                          dsLoMN + ((ks * 2048) >> 4), idDQ, ks > 0);
            tc_commit(&sh.dq_full[b]);
            #pragma unroll
            for (int ks = 0; ks < kBlockQ / 16; ++ks)
                mma_ts_lo(tmem + kColDV, tmem + kColS + b * kBlockQ + ks * 8,
                          dLoMN + ((ks * 2048) >> 4), idAcc, (ks > 0 || !first) ? 1u : 0u);
            tc_commit(&sh.pt_free[b]);
            #pragma unroll
            for (int ks = 0; ks < kBlockQ / 16; ++ks)
                mma_ss_lo(tmem + kColDK, dsLoK + ((ks * 32) >> 4), qLoMN + ((ks * 2048) >> 4), idAcc,
                          (ks > 0 || !first) ? 1u : 0u);
            tc_commit(&sh.qd_empty[s]);
            tc_commit(&sh.ds_free[b]);
        }
        tc_commit(&sh.kv_empty[set]); // K_j read by dQ^T
        tc_commit(&sh.acc_full);
    }
out:
    tc_commit(&sh.drain[1]);
    mbar_drain_wait(&sh.drain[1], 0);
}

// ---------------------------------------------------- softmax-gradient warps
// The elementwise pass for one key row, in steps of 16 queries:
//   P = 2^(s * scale * log2e - LSE * log2e),  dS = P * (dP - D),
// with -LSE*log2e and -D read as broadcast float4 rows, packed f32x2 math, and
// P, dS rounded to bf16 pairs.  Each step's Sᵀ and dPᵀ columns are loaded
// while the previous step computes (two register sets of 16 + 16 values);
// Pᵀ of a step goes over the Sᵀ columns of its own queries (already read),
// dSᵀ into the step's two 16-byte chunks of the key's row (chunk index XOR
// (row & 7), the 128-byte swizzle).  EDGE: queries outside [lo_c, hi_c)
// take P = 0, as a select, so the unrolled code has no branches.
template <bool EDGE>
__device__ __forceinline__ bool grad_row(uint32_t tS, uint32_t tdP, const float4 *nl4,
                                         const float4 *nd4, uint64_t c2, int lo_c, int hi_c,
                                         uint8_t *dsb, int r, uint64_t *ds_free, uint32_t ds_par,
                                         bool wait_ds, volatile int *abort) {
    uint32_t sr[2][kPartQ], dr[2][kPartQ];
    tmem_ld16(tS, sr[0]);
    tmem_ld16(tdP, dr[0]);
    tmem_wait_ld();
    #pragma unroll
    for (int qi = 0; qi < kBlockQ / kPartQ; ++qi) {
        const int cur = qi & 1;
        if (qi + 1 < kBlockQ / kPartQ) {
            tmem_ld16(tS + (qi + 1) * kPartQ, sr[cur ^ 1]);
            tmem_ld16(tdP + (qi + 1) * kPartQ, dr[cur ^ 1]);
        }
        uint32_t pk[kPartQ / 2], dk[kPartQ / 2];
        #pragma unroll
        for (int cc = 0; cc < kPartQ; cc += 4) {
            const int c = qi * kPartQ + cc;
            const float4 nl = nl4[c >> 2], nd = nd4[c >> 2];
            float x0, x1, x2, x3;
            f2unpack(f2fma(f2pack(__uint_as_float(sr[cur][cc]), __uint_as_float(sr[cur][cc + 1])), c2,
                           f2pack(nl.x, nl.y)), x0, x1);
            f2unpack(f2fma(f2pack(__uint_as_float(sr[cur][cc + 2]), __uint_as_float(sr[cur][cc + 3])), c2,
                           f2pack(nl.z, nl.w)), x2, x3);
            float p0 = ex2(x0), p1 = ex2(x1), p2 = ex2(x2), p3 = ex2(x3);
            if constexpr (EDGE) {
                p0 = (c + 0 >= lo_c && c + 0 < hi_c) ? p0 : 0.f;
                p1 = (c + 1 >= lo_c && c + 1 < hi_c) ? p1 : 0.f;
                p2 = (c + 2 >= lo_c && c + 2 < hi_c) ? p2 : 0.f;
                p3 = (c + 3 >= lo_c && c + 3 < hi_c) ? p3 : 0.f;
            }
            float d0, d1, d2, d3;
            f2unpack(f2mul(f2pack(p0, p1),
                           f2add(f2pack(__uint_as_float(dr[cur][cc]), __uint_as_float(dr[cur][cc + 1])),
                                 f2pack(nd.x, nd.y))), d0, d1);
            f2unpack(f2mul(f2pack(p2, p3),
                           f2add(f2pack(__uint_as_float(dr[cur][cc + 2]), __uint_as_float(dr[cur][cc + 3])),
                                 f2pack(nd.z, nd.w))), d2, d3);
            pk[cc >> 1] = pack_bf16(p0, p1);
            pk[(cc >> 1) + 1] = pack_bf16(p2, p3);
            dk[cc >> 1] = pack_bf16(d0, d1);
            dk[(cc >> 1) + 1] = pack_bf16(d2, d3);
        }
        tmem_st8(tS + qi * (kPartQ / 2), pk);
        // dK and dQ^T of tile n-2 read this dSᵀ buffer
        if (qi == 0 && wait_ds && !mbar_wait_warp(ds_free, ds_par, abort)) {
            tmem_wait_ld();     // the next step's load is in flight
            return false;
        }
        #pragma unroll
        for (int c2i = 0; c2i < 2; ++c2i) {
            const int ch = qi * 2 + c2i;
            const uint4 v = make_uint4(dk[4 * c2i], dk[4 * c2i + 1], dk[4 * c2i + 2], dk[4 * c2i + 3]);
            *reinterpret_cast<uint4 *>(dsb + ((ch ^ (r & 7)) << 4)) = v;
        }
        if (qi + 1 < kBlockQ / kPartQ) tmem_wait_ld();
    }
    return true;
}

template <int DH, bool CROSS>
__device__ void softmax_wg(const Params &p, Shared &sh, uint8_t *smem) {
    volatile int *abort = &sh.abort;
    const int warp = warp_id(), lane = lane_id();
    const int wg = warp >> 2;                  // takes tiles n with n % 2 == wg
    const int r = (warp & 3) * 32 + lane;      // key row of the block
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = sh.tmem_base + lanes + kColS + wg * kBlockQ;
    const uint32_t tdP = sh.tmem_base + lanes + kColDP + wg * kBlockQ;
    const float *rows = reinterpret_cast<const float *>(smem + kOffRows<DH>);
    uint8_t *dsb = smem + kOffDS + wg * kDSBytes + r * 128;
    const float sl2 = p.scale_log2;
    uint32_t n = 0, uc = 0;

    FOR_EACH_BWD_UNIT(u) {
        Unit w;
        const bool any = get_unit<CROSS>(u, p, w);
        const int kj = w.j0 + r;                  // this thread's key
        uint16_t *dst = static_cast<uint16_t *>(wg ? p.dk : p.dv) +
                        ((size_t)(w.tokk0 + kj) * p.Hkv + w.kvh) * DH;
        if (CROSS && w.last) {
            // keys that no query sees
            for (int i = (any ? w.Lk : 0) + r; i < w.Ls; i += kBlockK) {
                uint16_t *row = static_cast<uint16_t *>(wg ? p.dk : p.dv) +
                                ((size_t)(w.tokk0 + i) * p.Hkv + w.kvh) * DH;
                #pragma unroll
                for (int c = 0; c < DH; c += 8)
                    *reinterpret_cast<uint4 *>(row + c) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        if (!any) continue;
        const bool key_ok = kj < w.Lk;
        for (int k = 0; k < w.ntiles; ++k, ++n) {
            if ((int)(n & 1) != wg) continue;
            const int s = n % kStages<DH>;
            if (!mbar_wait_warp(&sh.s_full[wg], (n >> 1) & 1, abort)) return;
            if (!mbar_wait_warp(&sh.qd_full[s], (n / kStages<DH>) & 1, abort)) return;
            tc_fence_after();
            int h, q0;
            tile_of(w, p, k, h, q0);
            (void)h;
            const float4 *nl4 = reinterpret_cast<const float4 *>(rows + s * 2 * kBlockQ);
            const float4 *nd4 = nl4 + kBlockQ / 4;
            const int qmax = min(q0 + kBlockQ, w.L) - 1;
            const bool edge = (w.j0 + kBlockK > w.Lk) || (p.causal && w.jl > q0) ||
                              (p.window > 0 && w.j0 <= qmax - p.window);
            // The mask of an edge tile: the column range [lo_c, hi_c) of this
            // key's visible queries.
            int lo_c = 0, hi_c = kBlockQ;
            if (!key_ok) {
                lo_c = kBlockQ;
                hi_c = 0;
            } else if (p.causal) {
                lo_c = kj - q0;                                   // query >= key
                if (p.window > 0) hi_c = min(kBlockQ, kj + p.window - q0);   // query < key + W
            }
            const uint64_t c2 = f2pack(sl2, sl2);
            const bool ok = edge
                ? grad_row<true>(tS, tdP, nl4, nd4, c2, lo_c, hi_c, dsb, r, &sh.ds_free[wg],
                                 ((n - 2) >> 1) & 1, n >= 2, abort)
                : grad_row<false>(tS, tdP, nl4, nd4, c2, 0, 0, dsb, r, &sh.ds_free[wg],
                                  ((n - 2) >> 1) & 1, n >= 2, abort);
            if (!ok) return;
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[wg]);
        }
        // ---- unit end: warpgroup 0 writes dV, warpgroup 1 writes scale * dK
        if (!mbar_wait_warp(&sh.acc_full, uc & 1, abort)) return;
        ++uc;
        tc_fence_after();
        const uint32_t tAcc = sh.tmem_base + lanes + (wg ? kColDK : kColDV);
        const float mul = wg ? p.scale : 1.f;
        #pragma unroll
        for (int c = 0; c < DH; c += 32) {
            uint32_t v[32];
            tmem_ld32(tAcc + c, v);
            tmem_wait_ld();
            if (key_ok) {
                uint4 *d4 = reinterpret_cast<uint4 *>(dst + c);
                #pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint4 o;
                    o.x = pack_bf16(__uint_as_float(v[8 * e + 0]) * mul, __uint_as_float(v[8 * e + 1]) * mul);
                    o.y = pack_bf16(__uint_as_float(v[8 * e + 2]) * mul, __uint_as_float(v[8 * e + 3]) * mul);
                    o.z = pack_bf16(__uint_as_float(v[8 * e + 4]) * mul, __uint_as_float(v[8 * e + 5]) * mul);
                    o.w = pack_bf16(__uint_as_float(v[8 * e + 6]) * mul, __uint_as_float(v[8 * e + 7]) * mul);
                    d4[e] = o;
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.acc_free);
    }
}

// ------------------------------------------------------------- dQ drain
// dQ^T of a tile (lane = d index, column = query) is read from TMEM, scaled,
// written transposed into a shared-memory staging buffer (32 query rows x d,
// fp32) and added into the global accumulator by one TMA reduce-add per 32
// rows; two staging buffers alternate so the next rows are written while the
// previous reduce still reads.  Rows past the sequence add exact zeros (their
// P, hence dS, is 0).
template <int DH, bool CROSS>
__device__ void dq_drain(const CUtensorMap *tmDQ, const Params &p, Shared &sh, uint8_t *smem) {
    volatile int *abort = &sh.abort;
    const int warp = warp_id(), lane = lane_id();
    const int c = (warp & 3) * 32 + lane;       // d index (TMEM lane of dQ^T)
    const bool leader = (warp == kWarpDrain && lane == 0);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    float *stage = reinterpret_cast<float *>(smem + kOffDQ);
    uint32_t n = 0, hs = 0;
    FOR_EACH_BWD_UNIT(u) {
        Unit w;
        if (!get_unit<CROSS>(u, p, w)) continue;
        for (int k = 0; k < w.ntiles; ++k, ++n) {
            const int b = n & 1;
            const bool ok = mbar_wait_warp(&sh.dq_full[b], (n >> 1) & 1, abort);
            if (!named_bar_and(kBarDrain, 128, ok)) goto out;
            tc_fence_after();
            uint32_t v[64];
            const uint32_t t = sh.tmem_base + lanes + kColDP + b * kBlockQ;
            tmem_ld32(t, v);
            tmem_ld32(t + 32, v + 32);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.dq_free[b]);
            int h, q0;
            tile_of(w, p, k, h, q0);
            #pragma unroll
            for (int half = 0; half < 2; ++half, ++hs) {
                float *buf = stage + (hs & 1) * (kDQHalf * kD);
                if (leader) bulk_wait_group_read<1>();   // the reduce that used buf is done reading
                named_bar_sync(kBarDrain, 128);
                if (c < DH) {           // rows of the head dim (the reduce box is DH wide)
                    #pragma unroll
                    for (int i = 0; i < kDQHalf; ++i)
                        buf[i * DH + c] = __uint_as_float(v[half * kDQHalf + i]) * p.scale;
                }
                fence_proxy_async_smem();
                named_bar_sync(kBarDrain, 128);
                if (leader) {
                    tma_reduce_add_3d(tmDQ, buf, 0, h, w.tok0 + q0 + half * kDQHalf);
                    bulk_commit_group();
                }
            }
        }
    }
out:
    if (leader) bulk_wait_group_all();
}

template <int DH, bool CROSS>
__global__ void __launch_bounds__(kThreads, 1)
bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
           const __grid_constant__ CUtensorMap tmDQ, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    const uint32_t base = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024 - (base & 1023)) & 1023);
    const int warp = warp_id();

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages<DH>; ++s) {
            mbar_init(&sh.qd_full[s], 2);   // TMA bytes + the LSE/D rows
            mbar_init(&sh.qd_empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.s_full[b], 1);
            mbar_init(&sh.p_full[b], 4);
            mbar_init(&sh.dq_full[b], 1);
            mbar_init(&sh.dq_free[b], 4);
            mbar_init(&sh.pt_free[b], 1);
            mbar_init(&sh.ds_free[b], 1);
            mbar_init(&sh.kv_full[b], 1);
            mbar_init(&sh.kv_empty[b], 2);  // one commit from each MMA issuer
        }
        mbar_init(&sh.acc_full, 1);
        mbar_init(&sh.acc_free, 8);
        mbar_init(&sh.drain[0], 1);
        mbar_init(&sh.drain[1], 1);
        mbar_init(&sh.kv_tail, 1);
        mbar_init(&sh.qd_tail, 1);
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == kWarpMma) tmem_alloc(&sh.tmem_base, kTmemCols);
    if (warp == kWarpTma && lane_id() == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        tma_prefetch_desc(&tmdO);
        tma_prefetch_desc(&tmDQ);
    }
    if constexpr (CROSS) {
        // before the tiles or behind them: of the 1,024 bytes that align them
        // one part holds 512
        const int front = (int)(smem - smem_raw);
        DealTable *deal = reinterpret_cast<DealTable *>(front >= 512 ? smem_raw : smem + kSmemBytes - 1024);
        if (threadIdx.x == 0) sh.deal = deal;
        deal_begin(*deal, p.num_seqs, p.Hkv, CrossUnits{p});
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    if (warp < 8) {
        regs_increase<kRegsSoftmax>();
        softmax_wg<DH, CROSS>(p, sh, smem);
    } else if (warp < 12) {
        regs_decrease<kRegsDrain>();
        dq_drain<DH, CROSS>(&tmDQ, p, sh, smem);
    } else {
        regs_decrease<kRegsControl>();
        if (warp == kWarpTma) {
            producer<DH, CROSS>(&tmQ, &tmK, &tmV, &tmdO, p, sh, smem);
        } else if (warp == kWarpMma) {
            if (lane_id() == 0) mma_issuer_s<DH, CROSS>(p, sh, smem);
        } else if (warp == kWarpMmaGrad) {
            if (lane_id() == 0) mma_issuer_grad<DH, CROSS>(p, sh, smem);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(sh.tmem_base, kTmemCols);
    }
}

// D = rowsum(O * dO) for every (token, query head), in the LSE layout; zeroes
// the dQ accumulator.  A warp takes kPrepRows rows of DH = 64 or 128 elements,
// all their loads first (one row's would leave HBM waiting), and four lanes
// work out where the four results go, with one division for all of them:
// 13.5 us for 27.6 a row at a time (24 x 1,024 queries at most, 16 heads,
// d = 64), 17.7 for 26.1 (4,096, 32 heads, d = 128).
constexpr int kPrepRows = 4;

template <int DH>
__global__ void __launch_bounds__(256)
bwd_prep_kernel(const uint16_t *__restrict__ o, const uint16_t *__restrict__ dout,
                float *__restrict__ dd, float *__restrict__ dq_acc, int total, int Hq,
                int seqlen, int dense) {
    const long long row0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kPrepRows;
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)total * Hq;
    if (row0 >= rows) return;
    const int n = (int)min((long long)kPrepRows, rows - row0);
    auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
    auto hi = [](uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); };
    using Load = std::conditional_t<DH == 128, uint2, uint32_t>;
    Load a[kPrepRows], b[kPrepRows];
    #pragma unroll
    for (int i = 0; i < kPrepRows; ++i) {
        a[i] = b[i] = Load{};
        if (i < n) {
            a[i] = reinterpret_cast<const Load *>(o + (row0 + i) * DH)[lane];
            b[i] = reinterpret_cast<const Load *>(dout + (row0 + i) * DH)[lane];
        }
    }
    float mine = 0.f;
    #pragma unroll
    for (int i = 0; i < kPrepRows; ++i) {
        float acc;
        if constexpr (DH == 128) {
            acc = lo(a[i].x) * lo(b[i].x) + hi(a[i].x) * hi(b[i].x) + lo(a[i].y) * lo(b[i].y) +
                  hi(a[i].y) * hi(b[i].y);
            if (i < n)
                reinterpret_cast<float4 *>(dq_acc + (row0 + i) * DH)[lane] = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
            acc = lo(a[i]) * lo(b[i]) + hi(a[i]) * hi(b[i]);
            if (i < n) reinterpret_cast<float2 *>(dq_acc + (row0 + i) * DH)[lane] = make_float2(0.f, 0.f);
        }
        #pragma unroll
        for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
        if (lane == i) mine = acc;
    }
    if (lane < n) {
        const long long row = row0 + lane;
        const long long tok = row / Hq;
        const int h = (int)(row % Hq);
        size_t idx;
        if (dense) {
            const long long bseq = tok / seqlen, i = tok % seqlen;
            idx = ((size_t)bseq * Hq + h) * seqlen + i;
        } else {
            idx = (size_t)h * total + tok;
        }
        dd[idx] = mine;
    }
}

// Gradient of a learned sink logit z_h: the sink is one more score with a
// zero value, so its dP is 0 and d Loss / d z_h = sum over the rows of head h
// of exp(z_h - LSE_i) * (0 - D_i).  One block per head; a fixed-order tree
// reduction (deterministic).
__global__ void __launch_bounds__(256)
bwd_dsink_kernel(const float *__restrict__ lse, const float *__restrict__ dd,
                 const float *__restrict__ sinks, float *__restrict__ dsinks, int num_seqs,
                 int Hq, int seqlen, int total, int dense) {
    const int h = blockIdx.x;
    const float z = sinks[h];
    float acc = 0.f;
    if (z != -INFINITY) {
        const long long rows = dense ? (long long)num_seqs * seqlen : total;
        for (long long r = threadIdx.x; r < rows; r += blockDim.x) {
            size_t idx;
            if (dense)
                idx = ((size_t)(r / seqlen) * Hq + h) * seqlen + (r % seqlen);
            else
                idx = (size_t)h * total + r;
            acc -= __expf(z - lse[idx]) * dd[idx];
        }
    }
    #pragma unroll
    for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    __shared__ float part[8];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        float t = 0.f;
        for (int w = 0; w < 8; ++w) t += part[w];
        dsinks[h] = t;
    }
}

// dQ (bf16) = the fp32 accumulator, eight elements per thread.  With cu (cross
// attention, packed) only rows of the sequences, cu[0] .. cu[num_seqs]-1;
// per8: threads per token.
__global__ void __launch_bounds__(256)
bwd_convert_kernel(const float *__restrict__ acc, uint16_t *__restrict__ dq, long long n8,
                   const int *__restrict__ cu, int num_seqs, int per8) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n8) return;
    if (cu) {
        const long long t = i / per8;
        if (t < __ldg(cu) || t >= __ldg(cu + num_seqs)) return;
    }
    const float4 a = reinterpret_cast<const float4 *>(acc)[2 * i];
    const float4 b = reinterpret_cast<const float4 *>(acc)[2 * i + 1];
    uint4 o;
    o.x = pack_bf16(a.x, a.y);
    o.y = pack_bf16(a.z, a.w);
    o.z = pack_bf16(b.x, b.y);
    o.w = pack_bf16(b.z, b.w);
    reinterpret_cast<uint4 *>(dq)[i] = o;
}

// Cross attention without any query: zeros into the sequences' rows of dK and
// dV; per8 16-byte words per row.
__global__ void __launch_bounds__(256)
bwd_zero_kernel(uint4 *__restrict__ dk, uint4 *__restrict__ dv, const Params p, int per8) {
    for (int s = 0; s < p.num_seqs; ++s) {
        int tok0, L, tokk0, Lk, Ls;
        if (!cross_lengths(p, s, tok0, L, tokk0, Lk, Ls)) {
            if (blockIdx.x == 0 && threadIdx.x == 0) report_error(kDevErrInput);
            continue;
        }
        const long long first = (long long)tokk0 * per8, n = (long long)Ls * per8;
        for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += 256ll * gridDim.x) {
            dk[first + i] = make_uint4(0u, 0u, 0u, 0u);
            dv[first + i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

}  // namespace bwd_impl

size_t bwd_workspace_bytes(long long total_tokens, int Hq, int d) {
    if (total_tokens < 0 || Hq <= 0 || (d != 64 && d != 128)) return 0;
    const size_t acc = (size_t)total_tokens * Hq * d * sizeof(float);
    const size_t dd = (size_t)total_tokens * Hq * sizeof(float);
    return ((acc + 255) & ~(size_t)255) + ((dd + 255) & ~(size_t)255);
}

int launch_bwd(const BwdArgs &a, cudaStream_t stream) {
    using namespace bwd_impl;
    if (a.d != 64 && a.d != 128) return -2;
    const int dh = a.d;
    const long long total = a.total_tokens;
    if (a.num_seqs == 0) return 0;
    Params p{};
    p.lse = a.lse;
    p.dk = a.dk;
    p.dv = a.dv;
    p.cu_seqlens = a.cu_seqlens;
    p.num_seqs = a.num_seqs;
    p.seqlen = a.seqlen;
    p.total_tokens = (int)total;
    p.max_seqlen = a.max_seqlen;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.group = a.Hq / a.Hkv;
    p.causal = a.causal;
    p.window = a.causal ? a.window : 0;
    p.scale = a.scale;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.cu_seqlens_k = a.cu_seqlens_k;
    p.seq_lens_k = a.seq_lens_k;
    p.seqlen_k = a.seqlen_k;
    p.total_k = a.total_k;
    p.max_seqlen_k = a.max_seqlen_k;
    if (total == 0) {
        if (!a.cross || a.total_k == 0) return 0;
        bwd_zero_kernel<<<4 * device_sm_count(), 256, 0, stream>>>(
            static_cast<uint4 *>(a.dk), static_cast<uint4 *>(a.dv), p, a.Hkv * dh / 8);
        return cudaGetLastError() == cudaSuccess ? 0 : -5;
    }
    const size_t acc_bytes = ((size_t)total * a.Hq * dh * sizeof(float) + 255) & ~(size_t)255;
    float *dq_acc = static_cast<float *>(a.workspace);
    float *dd = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + acc_bytes);

    const long long rows = total * a.Hq;
    auto prep = dh == 128 ? bwd_prep_kernel<128> : bwd_prep_kernel<64>;
    prep<<<(unsigned)((rows + 8 * kPrepRows - 1) / (8 * kPrepRows)), 256, 0, stream>>>(
        static_cast<const uint16_t *>(a.o), static_cast<const uint16_t *>(a.dout), dd, dq_acc,
        (int)total, a.Hq, a.seqlen, a.cu_seqlens ? 0 : 1);
    if (cudaGetLastError() != cudaSuccess) return -5;
    if (a.sinks) {
        bwd_dsink_kernel<<<a.Hq, 256, 0, stream>>>(a.lse, dd, a.sinks, a.dsinks, a.num_seqs,
                                                   a.Hq, a.seqlen, (int)total,
                                                   a.cu_seqlens ? 0 : 1);
        if (cudaGetLastError() != cudaSuccess) return -5;
    }

    // Tiles are loaded in 64-column boxes: two of them for dh = 128, one for 64.
    alignas(64) CUtensorMap tq, tk, tv, tdo, tdq;
    const uint64_t T = (uint64_t)total;
    // (without any key the K and V maps are never used: any valid address)
    const bool no_keys = a.cross && a.total_k == 0;
    const uint64_t TK = no_keys ? 1 : a.cross ? (uint64_t)a.total_k : T;
    const void *k = no_keys ? a.q : a.k, *v = no_keys ? a.q : a.v;
    if (encode_tensor_map_3d(&tq, a.q, 2, dh, a.Hq, T, (uint64_t)dh * 2, (uint64_t)a.Hq * dh * 2,
                             64, 1, kBlockQ, 128) ||
        encode_tensor_map_3d(&tdo, a.dout, 2, dh, a.Hq, T, (uint64_t)dh * 2,
                             (uint64_t)a.Hq * dh * 2, 64, 1, kBlockQ, 128) ||
        encode_tensor_map_3d(&tk, k, 2, dh, a.Hkv, TK, (uint64_t)dh * 2,
                             (uint64_t)a.Hkv * dh * 2, 64, 1, kBlockK, 128) ||
        encode_tensor_map_3d(&tv, v, 2, dh, a.Hkv, TK, (uint64_t)dh * 2,
                             (uint64_t)a.Hkv * dh * 2, 64, 1, kBlockK, 128) ||
        encode_tensor_map_3d(&tdq, dq_acc, 4, dh, a.Hq, T, (uint64_t)dh * 4,
                             (uint64_t)a.Hq * dh * 4, dh, 1, kDQHalf, 0))
        return -5;
    p.dd = dd;
    p.dq_acc = dq_acc;
    // (cross attention: a unit at least per sequence, which finds lengths above the longest)
    p.num_kblocks = ((a.cross ? a.max_seqlen_k : a.max_seqlen) + kBlockK - 1) / kBlockK;
    if (a.cross && a.total_k > 0 && p.num_kblocks == 0) p.num_kblocks = 1;
    const long long units = (long long)p.num_kblocks * a.num_seqs * a.Hkv;
    if (units > (1ll << 30)) return -2;
    p.num_units = (int)units;
    if (units > 0) {
        auto kernel = a.cross ? (dh == 128 ? bwd_kernel<128, true> : bwd_kernel<64, true>)
                              : (dh == 128 ? bwd_kernel<128, false> : bwd_kernel<64, false>);
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmemBytes) != cudaSuccess)
            return -5;
        const int grid = (int)(units < device_sm_count() ? units : device_sm_count());
        kernel<<<grid, kThreads, kSmemBytes, stream>>>(tq, tk, tv, tdo, tdq, p);
        if (cudaGetLastError() != cudaSuccess) return -5;
    }
    const long long n8 = total * a.Hq * dh / 8;
    bwd_convert_kernel<<<(unsigned)((n8 + 255) / 256), 256, 0, stream>>>(
        dq_acc, static_cast<uint16_t *>(a.dq), n8, a.cross ? a.cu_seqlens : nullptr, a.num_seqs,
        a.Hq * dh / 8);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

}  // namespace fa
