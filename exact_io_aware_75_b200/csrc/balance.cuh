// balance.cuh -- ragged work dealt out evenly to a persistent grid.
//
// Sequences of different lengths give units of different cost; dealt out to
// 148 CTAs as they come, the busiest ends well after the average.  Here the
// sequences are ordered by the cost of their units first, dearest first, and
// the units dealt in rows of gridDim.x, in alternating directions: units of a
// row cost nearly the same, and CTAs at work at the same time share a sequence
// and its keys.  (Equal contiguous parts of the units, the other way, were 11 %
// slower on equal lengths.)  Each CTA orders the sequences for itself.  More
// than kDealSeqs of them are dealt as they come, which costs where they are
// short: 101 pairs of 10 to 200 queries on 20 to 400 keys take 142 us forward
// and 486 backward where 100 take 123 and 359 (32/8 heads, d = 128; 16/16 heads,
// d = 64: 85 and 223, 88 and 205).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "sm100.cuh"

namespace fa {

constexpr int kDealSeqs = 100;

// The units of one head of a sequence: how many, and the cost of the first.
struct SeqUnits {
    int n, cost;
};

struct DealTable {
    int first[kDealSeqs + 1];       // units before each sequence, in order
    uint8_t order[kDealSeqs];
};
static_assert(sizeof(DealTable) <= 512, "the backward finds it 512 bytes");

// All threads of a block of at least kDealSeqs; ends with a barrier.
template <class F>
__device__ __forceinline__ void deal_begin(DealTable &t, int num_seqs, int heads, F units) {
    if (num_seqs > kDealSeqs) return;
    const int s = threadIdx.x;
    SeqUnits c{0, 0};
    if (s < num_seqs) {
        c = units(s);
        t.first[s] = c.n > 0 ? c.cost : -1;
    }
    __syncthreads();
    int rank = 0;
    if (s < num_seqs) {
        const int mine = t.first[s];
        #pragma unroll 1
        for (int i = 0; i < num_seqs; ++i) {
            const int x = t.first[i];
            rank += x > mine || (x == mine && i < s);
        }
    }
    __syncthreads();
    if (s < num_seqs) {
        t.order[rank] = (uint8_t)s;
        t.first[rank + 1] = c.n * heads;
    }
    if (s == 0) t.first[0] = 0;
    __syncthreads();
    if (s < 32) {
        int running = 0;
        #pragma unroll 1
        for (int i0 = 1; i0 <= num_seqs; i0 += 32) {
            const int i = i0 + s;
            int x = i <= num_seqs ? t.first[i] : 0;
            #pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (s >= o) x += y;
            }
            if (i <= num_seqs) t.first[i] = running + x;
            running += __shfl_sync(0xffffffffu, x, 31);
        }
    }
    __syncthreads();
}

// The units of this CTA, for each thread that walks them: sequence, head and
// place in the head.  Only `it` and `r` live across a unit.
struct DealWalk {
    int it = 0, r = 0, s, h, k;
    __device__ __forceinline__ bool more(const DealTable &t, int num_seqs, int heads, int most) {
        const int g = gridDim.x, i = blockIdx.x;
        int u = (it & 1) ? (it + 1) * g - 1 - i : it * g + i;
        if (num_seqs <= kDealSeqs) {
            if (u >= t.first[num_seqs]) return false;     // (only the last row is short)
            while (u >= t.first[r + 1]) ++r;
            s = t.order[r];
            u -= t.first[r];
            k = u / heads;
            h = u - k * heads;
        } else {
            const int per = num_seqs * heads;
            k = u / per;
            if (k >= most) return false;
            u -= k * per;
            s = u / heads;
            h = u - s * heads;
        }
        return true;
    }
};

}  // namespace fa
