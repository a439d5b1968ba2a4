// delta_launch.hpp -- enqueue the gated delta rule's kernels on a stream.
#pragma once

#include "delta.hpp"

namespace ssd {
namespace delta {

// Waves of a work-group of k_delta and k_delta_rev, 16 columns of headdim each: as many as P allows, up
// to 4, and fewer while that leaves CUs without a work-group (float32, dstate 64, 512 tokens, 8 heads of
// 64: forward 78 us with one wave, 81 with four; backward 199, 211).
inline int walk_waves(int64_t bh, int64_t P) {
    int w = (int)(P / 16);
    if (w > 4) w = 4;
    while (w > 1 && bh * (P / (16 * w)) < 256) w >>= 1;
    return w;
}

// Shares of a group's heads in the gradient kernel: enough work-groups for every CU twice over, each
// summing as many heads in registers as that leaves.  Backward with 256 / 512 / 1024 / 2048 work-groups
// at least (us): 2 rows of 2048 tokens, 48 heads of 64, dstate 128: 556 / 509 / 520 / 535; one row of 4096,
// 128 heads: 1237 / 1111 / 1122 / 1135; one row of 2048, 32 heads of 128, dstate 256, 2 groups: 490 / 438 / 448
// / 467.
inline int grad_shares(int64_t chunks, int64_t H, int64_t G, int64_t N) {
    const int64_t base = chunks * G * (N > 64 ? N / 64 : 1), hg = H / G;
    int64_t s = (512 + base - 1) / (base > 0 ? base : 1);
    return (int)(s < 1 ? 1 : s > hg ? hg : s);
}

// Heads of a group that one work-group of the decays' gradients takes, sharing its Q K^T and K
// K^T: up to 4 while that leaves six work-groups per CU (backward of 2 rows of 2048 tokens, 48 heads:
// one head 530 us, two 521, three 520, four, with three work-groups per CU, 529).
inline int ddt_heads(int64_t ntab, int64_t H, int64_t G) {
    int s = 4;
    while (s > 1 && (s > H / G || ntab * G * ((H / G + s - 1) / s) < 1536)) s >>= 1;
    return s;
}

inline bool dma_walk(bool bf16_dtype, int64_t N);
inline int team_tiles(int64_t bh, int64_t P, int64_t N);
// Slices of headdim that the backward's walks write partial sums for, per token and (waves) per state.
inline int64_t bwd_slices(bool bf16_dtype, int64_t bh, int64_t P, int64_t N) {
    return P / (16 * (dma_walk(bf16_dtype, N) ? team_tiles(bh, P, N) : walk_waves(bh, P)));
}
inline int64_t bwd_tots(bool bf16_dtype, int64_t bh, int64_t P, int64_t N) {
    return dma_walk(bf16_dtype, N) ? 4 * bwd_slices(bf16_dtype, bh, P, N) : P / 16;
}

template <typename K>
bool lds_limit(K* kernel, size_t bytes) {
    return bytes <= 64 * 1024 || hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                                     (int)bytes) == hipSuccess;
}

template <typename T, int N>
int walk(const Args& a, int which) {
    typedef Cfg<T, N> CF;
    const int waves = walk_waves((int64_t)a.rows.nrows * a.H, a.P), sw = 16 * waves;
    const unsigned grid = (unsigned)((int64_t)a.rows.nrows * a.H * (a.P / sw));
    if (which == 0) {
        const size_t lds = CF::walk_bytes(sw, CF::NT > 1 ? 2 : 1, 1);
        if (!lds_limit(k_delta<T, N, false>, lds)) return 7;
        k_delta<T, N, false><<<grid, 256, lds, a.stream>>>(a, waves);
    } else if (which == 1) {
        const size_t lds = CF::walk_bytes(sw, 0, 2);
        if (!lds_limit(k_delta<T, N, true>, lds)) return 7;
        k_delta<T, N, true><<<grid, 256, lds, a.stream>>>(a, waves);
    } else {
        const size_t lds = CF::walk_bytes(sw, CF::NT, 2);
        if (!lds_limit(k_delta_rev<T, N>, lds)) return 7;
        k_delta_rev<T, N><<<grid, 256, lds, a.stream>>>(a, waves);
    }
    return hipGetLastError() == hipSuccess ? 0 : 7;
}

// Whether the walks run on tables stored as fragments (k_delta_dma, k_delta_team, k_delta_adj).
inline bool dma_walk(bool bf16_dtype, int64_t N) { return bf16_dtype && N >= 64; }

// Heads of a group that one wave of the preparation takes, sharing their K K^T and Q K^T: up to 4
// while that leaves four waves per SIMD.  Forward with 1 / 2 / 4 (us), 80 heads of 64, dstate 128: 8 rows of
// 4096 tokens (10240 waves with 4) 974 / 900 / 878, of 1024 (5120 with 2) 293 / 269 / 276; one row of 2048 tokens, 32
// heads (1024 with 1) 77 / 84 / 93.
inline int prep_heads(int64_t ntab, int64_t H, int64_t G) {
    int s = 4;
    while (s > 1 && (s > H / G || ntab * G * ((H / G + s - 1) / s) < 4096)) s >>= 1;
    return s;
}
template <typename T, int N, Tab TAB>
void prep(const Args& a) {
    const int heads = prep_heads(a.ntab, a.H, a.G);
    const int64_t waves = (int64_t)a.ntab * a.G * ((a.H / a.G + heads - 1) / heads);
    k_delta_prep<T, N, TAB><<<(unsigned)((waves + 3) / 4), 256, 0, a.stream>>>(a, heads);
}

template <int N, int KB, int OCC>
int walk_dma(const Args& a, int waves) {
    const unsigned grid = (unsigned)((int64_t)a.rows.nrows * a.H * (a.P / (16 * waves)));
    k_delta_dma<N, KB, OCC><<<grid, 64 * waves, 0, a.stream>>>(a);
    return hipGetLastError() == hipSuccess ? 0 : 7;
}
// Column tiles per team: one, or two where that still gives every CU a team (the key and table
// fragments are then read once for both; at dstate 256 LDS leaves no room).  2048 tokens, one / two tiles
// (us), headdim 64, dstate 128: 64 heads forward 89 / 107, backward 367 / 435; 96 heads 151 / 118, 623 / 519;
// headdim 32: 128 heads 98 / 120, 429 / 491; 192 heads 165 / 135, 719 / 606.
inline int team_tiles(int64_t bh, int64_t P, int64_t N) { return N <= 128 && P >= 32 && bh * P > 256 * 16 ? 2 : 1; }
template <int N, int CT, bool SAVE>
int walk_team(const Args& a) {
    const unsigned grid = (unsigned)((int64_t)a.rows.nrows * a.H * (a.P / (16 * CT)));
    // (at dstate 256 the backward's first walk is faster with one K buffer: 32 heads of 64, 4096 tokens, backward
    // 739 us, with two 761)
    k_delta_team<N, CT, N == 256 && SAVE ? 1 : 2, SAVE><<<grid, 512, 0, a.stream>>>(a);
    return hipGetLastError() == hipSuccess ? 0 : 7;
}
template <int N, int CT>
int walks_bwd(const Args& a) {
    const int st = walk_team<N, CT, true>(a);
    if (st) return st;
    const unsigned grid = (unsigned)((int64_t)a.rows.nrows * a.H * (a.P / (16 * CT)));
    k_delta_adj<N, CT, N == 256 ? 1 : 2><<<grid, 256, 0, a.stream>>>(a);
    return hipGetLastError() == hipSuccess ? 0 : 7;
}
// Teams while there are at most two column tiles a CU, and at any number of chains where a head is too
// narrow for a work-group of four waves to share its tables; else a wave per 16 columns.  Forward of
// 2048 tokens, whole call (us, team / wave): headdim 64, dstate 128: 32 heads 78 / 137, 128 heads 125 / 157, 192
// heads 214 / 177, 768 heads 653 / 515; dstate 256: 64 heads 116 / 205, 128 heads 219 / 228, 192 heads 319 / 256;
// headdim 128, dstate 128: 64 heads 105 / 145, 96 heads 191 / 157; headdim 32, dstate 128: 256 heads 158 / 188,
// 768 heads 425 / 430, 1536 heads 805 / 774; dstate 256: 256 heads 258 / 279, 1536 heads 1274 / 1376; headdim 16:
// 1536 heads, dstate 128 631 / 712, dstate 256 795 / 1582.
inline bool team_walk(int64_t bh, int64_t P, int64_t N) {
    return P < (N <= 128 ? 32 : 64) || bh * P <= 2 * 256 * 16;
}

template <typename T, int N>
int run_fwd(const Args& a) {
    if constexpr (std::is_same<T, bf16>::value && N >= 64) {
        prep<T, N, kFold>(a);
        const int64_t bh = (int64_t)a.rows.nrows * a.H;
        if (team_walk(bh, a.P, N)) {
            if constexpr (N <= 128) {
                if (team_tiles(bh, a.P, N) == 2) return walk_team<N, 2, false>(a);
            }
            return walk_team<N, 1, false>(a);
        }
        const int waves = a.P >= 64 ? 4 : 2;
        // As many work-groups per CU as LDS takes: three with one K buffer to dstate 64; two, with
        // two K buffers, at 128 (three, with the second term of M from memory: 24 ragged prompts 278
        // us against 260, the 2.7B layer shape 879 against 885); one at 256.
        return walk_dma<N, N <= 64 ? 1 : 2, N <= 64 ? 3 : N <= 128 ? 2 : 1>(a, waves);
    } else {
        prep<T, N, kPlain>(a);
        return walk<T, N>(a, 0);
    }
}

template <typename T>
void ddt(const Args& a) {
    const int heads = ddt_heads(a.ntab, a.H, a.G);
    const unsigned grid = (unsigned)((int64_t)a.ntab * a.G * ((a.H / a.G + heads - 1) / heads));
    if (a.P == 16) k_delta_ddt<T, 16><<<grid, 256, 0, a.stream>>>(a, heads);
    else if (a.P == 32) k_delta_ddt<T, 32><<<grid, 256, 0, a.stream>>>(a, heads);
    else k_delta_ddt<T, 64><<<grid, 256, 0, a.stream>>>(a, heads);
}

template <typename T, int N>
int run_bwd(const Args& a) {
    typedef GradCfg<T, N> GC;
    int st;
    if constexpr (std::is_same<T, bf16>::value && N >= 64) {
        prep<T, N, kBoth>(a);
        if constexpr (N <= 128) {
            st = team_tiles((int64_t)a.rows.nrows * a.H, a.P, N) == 2 ? walks_bwd<N, 2>(a) : walks_bwd<N, 1>(a);
        } else {
            st = walks_bwd<N, 1>(a);
        }
    } else {
        prep<T, N, kPlain>(a);
        st = walk<T, N>(a, 1);
        if (!st) st = walk<T, N>(a, 2);
    }
    if (st) return st;
    const size_t lds = GC::BYTES;
    if (!lds_limit(k_delta_grad<T, N>, lds)) return 7;
    const int64_t wgs = (int64_t)a.ntab * a.G * a.nsub * (N / GC::NS);
    k_delta_grad<T, N><<<(unsigned)wgs, 256, lds, a.stream>>>(a);
    if (a.nsub > 1) {
        const int64_t all = (int64_t)a.rows.nrows * a.T * a.G * N;
        k_delta_sum<T><<<(unsigned)((2 * all / 4 + 255) / 256), 256, 0, a.stream>>>(
            a.part, static_cast<T*>(a.dB), static_cast<T*>(a.dC), all, a.nsub);
    }
ddt<T>(a);
        k_delta_dA<64><<<(unsigned)a.H, 64, 0, a.stream>>>(a.dAp, a.dA, a.ntab, a.H);
    return hipGetLastError() == hipSuccess ? 0 : 7;
}

template <typename T>
int run(const Args& a, bool bwd) {
    switch (a.N) {
        case 16: return bwd ? run_bwd<T, 16>(a) : run_fwd<T, 16>(a);
        case 32: return bwd ? run_bwd<T, 32>(a) : run_fwd<T, 32>(a);
        case 64: return bwd ? run_bwd<T, 64>(a) : run_fwd<T, 64>(a);
        case 128: return bwd ? run_bwd<T, 128>(a) : run_fwd<T, 128>(a);
        case 256: return bwd ? run_bwd<T, 256>(a) : run_fwd<T, 256>(a);
        default: return 3;
    }
}

int run_bf16(const Args& a, bool bwd);
int run_f32(const Args& a, bool bwd);

}  // namespace delta
}  // namespace ssd
