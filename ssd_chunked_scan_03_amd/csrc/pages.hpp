// pages.hpp -- the pages of a pool of states (a page is a slot: one sequence's state in every
// layer): fork, free and begin by a table of sources, and compaction.
#pragma once

#include "device.hpp"

namespace ssd {
namespace pool {

// ---------------------------------------------------------------------------
// The pool's pages.  Every work-group forms the same plan from the table in LDS (it is a function of
// the table alone, and no work-group writes what another one's plan reads), then takes its share of
// the moves.  Sources and destinations of the moves are different slots, so their order is free.
// ---------------------------------------------------------------------------
constexpr int kSlots = 16384;     // slots of a pool at most
constexpr int kPiece = 256 * 4 * 8;  // floats of a move that one work-group copies at a time

struct PageArgs {
    int64_t layers, elems, ls, ss;
    int R, S;
    float* pool;
    const int* table;
    const int* sources;
    int* fresh;  // the new table
    int* count;
    hipStream_t stream;
};

// Set bits of words[0 .. n) before word w, for every w: `before` gets n + 1 counts.
__device__ __forceinline__ void count_bits(const unsigned long long* words, int* before, int n) {
    if (threadIdx.x < 64) {
        int run = 0;
        for (int w0 = 0; w0 < n; w0 += 64) {
            const int w = w0 + threadIdx.x, c = w < n ? __popcll(words[w]) : 0;
            int s = c;
            for (int off = 1; off < 64; off <<= 1) {
                const int v = __shfl_up(s, off, 64);
                if ((int)threadIdx.x >= off) s += v;
            }
            if (w < n) before[w] = run + s - c;
            run += __shfl(s, 63, 64);
        }
        if (threadIdx.x == 0) before[n] = run;
    }
    __syncthreads();
}
// The position of set bit number k (from 0): the last word that starts at or below it, then its bit.
__device__ __forceinline__ int nth_bit(const unsigned long long* words, const int* before, int n, int k) {
    int lo = 0, hi = n;  // before[lo] <= k < before[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= k) lo = mid;
        else hi = mid;
    }
    unsigned long long v = words[lo];
    for (int r = k - before[lo]; r > 0; --r) v &= v - 1;
    return lo * 64 + __ffsll((long long)v) - 1;
}

// Elements [at, at + kPiece) of a slot in one layer from slot `from` (negative: zeros) to slot `to`.  Two
// loads in flight per thread, and stores that leave no copy in the caches (copies of 0.28 GB of states,
// a slot 2.6 MB in a layer: two 122 us, two without the hint 130, four 123, eight 155, one 155).  Over pools in turn that
// do not fit the last-level cache, 0.58 GB read and written take 108 us: 5.4 TB/s, a large copy's rate.
__device__ __forceinline__ void copy_piece(const PageArgs& a, int from, int to, int64_t layer, int64_t at) {
    constexpr int UN = 2;
    const float* src = a.pool + layer * a.ls + (int64_t)(from < 0 ? 0 : from) * a.ss;
    float* dst = a.pool + layer * a.ls + (int64_t)to * a.ss;
    for (int k0 = 0; k0 < kPiece; k0 += UN * 1024) {
        f32x4 v[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            const int64_t e = at + k0 + (k * 256 + threadIdx.x) * 4;
            v[k] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (from >= 0 && e < a.elems) v[k] = ld4(src + e);
        }
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            const int64_t e = at + k0 + (k * 256 + threadIdx.x) * 4;
            if (e < a.elems) __builtin_nontemporal_store(v[k], reinterpret_cast<f32x4*>(dst + e));
        }
    }
}

__global__ __launch_bounds__(256) void k_fork(PageArgs a) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int words = (a.S + 63) / 64, R = a.R, S = a.S;
    unsigned long long* free_ = reinterpret_cast<unsigned long long*>(smem);  // [words] slots that no row goes on from
    int* before = reinterpret_cast<int*>(free_ + words);                      // [words + 1]
    int* wave_n = before + words + 1;                                         // [4]
    int* owner = wave_n + 4;                                                  // [S] the row that takes the slot over
    unsigned* moves = reinterpret_cast<unsigned*>(owner + S);                 // [R] source (0xffff: zeros), destination
    constexpr int kNone = 0x7fffffff;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int s = tid; s < S; s += 256) owner[s] = kNone;
    for (int w = tid; w < words; w += 256) free_[w] = S - 64 * w >= 64 ? ~0ull : (1ull << (S - 64 * w)) - 1;
    __syncthreads();
    auto wanted = [&](int r) {
        const int q = a.sources[r];
        if (q < 0 || q >= R) return -1;
        const int s = a.table[q];
        return s >= 0 && s < S ? s : -1;
    };
    // (a row that keeps its own slot comes before all others)
    for (int r = tid; r < R; r += 256) {
        const int s = wanted(r);
        if (s < 0) continue;
        atomicMin(&owner[s], a.table[r] == s ? r : R + r);
        atomicAnd(&free_[s >> 6], ~(1ull << (s & 63)));
    }
    __syncthreads();
    count_bits(free_, before, words);
    int n = 0;  // moves so far
    for (int r0 = 0; r0 < R; r0 += 256) {
        const int r = r0 + tid;
        const int s = r < R ? wanted(r) : -1;
        const bool zero = r < R && a.sources[r] == -2;
        const bool takes = s >= 0 && owner[s] % R == r;
        const bool need = zero || (s >= 0 && !takes);
        const unsigned long long ask = __ballot(need);
        if (lane == 0) wave_n[wave] = __popcll(ask);
        __syncthreads();
        int at = n + __popcll(ask & ((1ull << lane) - 1));
        for (int w = 0; w < wave; ++w) at += wave_n[w];
        for (int w = 0; w < 4; ++w) n += wave_n[w];
        __syncthreads();
        int to = takes ? s : -1;
        if (need) {
            to = nth_bit(free_, before, words, at);
            moves[at] = (unsigned)(zero ? 0xffff : s) << 16 | (unsigned)to;
        }
        if (blockIdx.x == 0 && r < R) a.fresh[r] = to;
    }
    __syncthreads();
    const int64_t pieces = (a.elems + kPiece - 1) / kPiece, items = (int64_t)n * a.layers * pieces;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const unsigned m = moves[i / (a.layers * pieces)];
        const int64_t rest = i % (a.layers * pieces);
        copy_piece(a, m >> 16 == 0xffff ? -1 : (int)(m >> 16), (int)(m & 0xffff), rest / pieces, rest % pieces * kPiece);
    }
}

__global__ __launch_bounds__(256) void k_compact(PageArgs a) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int words = (a.S + 63) / 64, R = a.R, S = a.S;
    unsigned long long* live = reinterpret_cast<unsigned long long*>(smem);  // [words] slots that the table names
    unsigned long long* hole = live + words;                                 // [words] the others below their number
    int* before = reinterpret_cast<int*>(hole + words);                      // [words + 1] of live
    int* hbefore = before + words + 1;                                       // [words + 1] of hole
    const int tid = threadIdx.x;
    for (int w = tid; w < words; w += 256) live[w] = 0;
    __syncthreads();
    for (int r = tid; r < R; r += 256) {
        const int s = a.table[r];
        if (s >= 0 && s < S) atomicOr(&live[s >> 6], 1ull << (s & 63));
    }
    __syncthreads();
    count_bits(live, before, words);
    const int n = before[words];
    for (int w = tid; w < words; w += 256) {
        const int k = n - 64 * w;  // of this word's slots, those below n
        hole[w] = k <= 0 ? 0 : ~live[w] & (k >= 64 ? ~0ull : (1ull << k) - 1);
    }
    __syncthreads();
    count_bits(hole, hbefore, words);
    const int moves = hbefore[words];  // as many live slots at n and above as holes below it
    const int kept = n - moves;        // live slots below n
    if (blockIdx.x == 0) {
        for (int r = tid; r < R; r += 256) {
            int s = a.table[r];
            if (s < 0 || s >= S) s = -1;
            if (s >= n) {
                const int rank = before[s >> 6] + __popcll(live[s >> 6] & ((1ull << (s & 63)) - 1));
                s = nth_bit(hole, hbefore, words, rank - kept);
            }
            a.fresh[r] = s;
        }
        if (tid == 0) a.count[0] = n;
    }
    const int64_t pieces = (a.elems + kPiece - 1) / kPiece, items = (int64_t)moves * a.layers * pieces;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const int m = (int)(i / (a.layers * pieces));
        const int64_t rest = i % (a.layers * pieces);
        copy_piece(a, nth_bit(live, before, words, kept + m), nth_bit(hole, hbefore, words, m), rest / pieces,
                   rest % pieces * kPiece);
    }
}

inline size_t fork_lds(int64_t R, int64_t S) {
    const size_t words = (size_t)(S + 63) / 64;
    return words * 8 + (words + 1 + 4 + (size_t)S + (size_t)R) * 4;
}
inline size_t compact_lds(int64_t S) {
    const size_t words = (size_t)(S + 63) / 64;
    return words * 16 + 2 * (words + 1) * 4;
}
// Work-groups: one per piece of the most moves that there can be, up to four per CU or as many as LDS
// lets in (the copies above with 256 / 512 / 1024 / 2048 work-groups: 166 / 122 / 122 / 132 us; pieces of 8 / 16 / 32 / 64 KB:
// 122 / 125 / 122 / 128 us, and 152 / 123 / 113 / 114 us for a compaction of 0.27 GB in slots of 1.6 MB).
inline unsigned page_grid(const PageArgs& a, int64_t moves, size_t lds) {
    int64_t most = 256 * (160 * 1024 / (int64_t)(lds > 40 * 1024 ? lds : 40 * 1024));
    const int64_t pieces = (a.elems + kPiece - 1) / kPiece;
    const int64_t each = pieces < most / (a.layers > 0 ? a.layers : 1) + 1 ? a.layers * pieces : most;
    const int64_t items = moves * each;
    if (items < most) most = items;
    return (unsigned)(most < 1 ? 1 : most);
}

}  // namespace pool
}  // namespace ssd
