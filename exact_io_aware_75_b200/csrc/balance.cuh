// balance.cuh -- equal shares of ragged work for a persistent grid.
//
// Sequences of different lengths give units of different cost: dealt out in
// turn, the busiest of 148 CTAs with seven units each ends a third later than
// the average (16 x 448 queries on 400 to 1,500 keys).  Here the units stand
// in one row, sequence by sequence, head by head, and a CTA takes those that
// begin in its part of the row's total cost.  No table and no limit on the
// number of sequences: a scan over the sequences finds the one a part begins
// in, and from there on the walk goes by the sequences' own lengths.
#pragma once

#include <cuda_runtime.h>

#include "sm100.cuh"

namespace fa {

// The units of one head of a sequence: n, all of cost `unit` but the last.
struct SeqCost {
    int n, unit, last;
    __device__ __forceinline__ long long head() const {
        return n > 0 ? (long long)(n - 1) * unit + last : 0;
    }
};

// A unit: its sequence, head and place in the head.
struct UnitAt {
    int s, h, k;
};

struct Balance {
    UnitAt first, end;     // this CTA's units: from `first` up to, not including, `end`
    long long warp[16];
};

// All threads of the block; ends with a barrier.
template <int THREADS, class F>
__device__ __forceinline__ void balance_begin(Balance &b, int num_seqs, int heads, F cost) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long total = 0;
    #pragma unroll 1
    for (int s = tid; s < num_seqs; s += THREADS) total += cost(s, true).head();
    #pragma unroll 1
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) b.warp[warp] = total;
    if (tid == 0) b.first = b.end = UnitAt{num_seqs, 0, 0};
    __syncthreads();
    total = 0;
    #pragma unroll 1
    for (int w = 0; w < THREADS / 32; ++w) total += b.warp[w];
    total *= heads;
    long long running = 0;
    #pragma unroll 1
    for (int s0 = 0; s0 < num_seqs; s0 += THREADS) {
        const int s = s0 + tid;
        const SeqCost c = s < num_seqs ? cost(s, false) : SeqCost{0, 0, 0};
        long long inc = c.head();
        #pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        __syncthreads();
        if (lane == 31) b.warp[warp] = inc;
        __syncthreads();
        long long before = running;
        #pragma unroll 1
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += b.warp[w];
            running += b.warp[w];
        }
        const long long head = c.head();
        before = (before + inc - head) * heads;
        // the bounds of this CTA's part that lie in this sequence
        #pragma unroll 1
        for (int e = 0; e < 2; ++e) {
            const long long g = gridDim.x, i = blockIdx.x + e;
            const long long off = total / g * i + total % g * i / g - before;
            if (head == 0 || off < 0 || off >= head * heads) continue;
            // the first unit that begins at or behind the bound
            UnitAt u{s, (int)(off / head), 0};
            u.k = (int)((off - u.h * head + c.unit - 1) / c.unit);
            if (u.k >= c.n) {
                u.k = 0;
                if (++u.h == heads) {
                    u.h = 0;
                    do ++u.s;
                    while (u.s < num_seqs && cost(u.s, false).n == 0);
                }
            }
            if (e) b.end = u; else b.first = u;
        }
    }
    __syncthreads();
}

// The units of this CTA's part, for each thread that walks them.  Three numbers
// are kept; the rest is worked out again at each step, since the walkers'
// inner loops have no registers to spare.
template <class F>
struct BalanceWalk : UnitAt {
    __device__ __forceinline__ explicit BalanceWalk(const Balance &b) : UnitAt(b.first) {}
    __device__ __forceinline__ bool more(const Balance &b) const {
        return s != b.end.s || h != b.end.h || k != b.end.k;
    }
    __device__ __forceinline__ void step(F cost, int num_seqs, int heads) {
        if (++k < cost(s, false).n) return;
        k = 0;
        if (++h < heads) return;
        h = 0;
        do ++s;
        while (s < num_seqs && cost(s, false).n == 0);
    }
};

}  // namespace fa
