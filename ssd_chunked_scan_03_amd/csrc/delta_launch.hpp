// delta_launch.hpp -- enqueue the gated delta rule's kernels on a stream.
#pragma once

#include "delta.hpp"

namespace ssd {
namespace delta {

// Columns of headdim one work-group of the chunk walks takes: waves of 16 CT columns.  Two
// column tiles per wave read each table and key fragment once for both (bfloat16, where the
// state's accumulators leave the registers for it); as many waves as P allows, up to 4.
struct Slice {
    int ct, waves;
    int cols() const { return 16 * ct * waves; }
};
inline Slice slice_of(bool bf16_dtype, int64_t bh, int64_t P, int64_t N) {
    Slice s;
    s.ct = bf16_dtype && N <= 128 && P >= 32 ? 2 : 1;
    s.waves = (int)(P / (16 * s.ct));
    if (s.waves > 4) s.waves = 4;
    while (s.waves > 1 && bh * (P / s.cols()) < 256) s.waves >>= 1;
    return s;
}

// Shares of a group's heads in the gradient kernel: enough work-groups for every CU several
// times over, each summing as many heads in registers as that leaves.
inline int grad_shares(int64_t chunks, int64_t H, int64_t G, int64_t N) {
    const int64_t base = chunks * G * (N > 64 ? N / 64 : 1), hg = H / G;
    int64_t s = (1024 + base - 1) / (base > 0 ? base : 1);
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
    return P / (dma_walk(bf16_dtype, N) ? 16 * team_tiles(bh, P, N) : slice_of(bf16_dtype, bh, P, N).cols());
}
inline int64_t bwd_tots(bool bf16_dtype, int64_t bh, int64_t P, int64_t N) {
    return bwd_slices(bf16_dtype, bh, P, N) * (dma_walk(bf16_dtype, N) ? 4 : slice_of(bf16_dtype, bh, P, N).waves);
}

template <typename K>
bool lds_limit(K* kernel, size_t bytes) {
    return bytes <= 64 * 1024 || hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                                     (int)bytes) == hipSuccess;
}

template <typename T, int N, int CT>
int walk(const Args& a, int waves, int which) {
    typedef Cfg<T, N> CF;
    const int sw = 16 * CT * waves;
    const unsigned grid = (unsigned)((int64_t)a.rows.nrows * a.H * (a.P / sw));
    if (which == 0) {
        const size_t lds = CF::walk_bytes(sw, CF::NT > 1 ? 2 : 1, 1);
        if (!lds_limit(k_delta<T, N, CT, false>, lds)) return 7;
        k_delta<T, N, CT, false><<<grid, 256, lds, a.stream>>>(a, waves);
    } else if (which == 1) {
        const size_t lds = CF::walk_bytes(sw, 0, 2);
        if (!lds_limit(k_delta<T, N, CT, true>, lds)) return 7;
        k_delta<T, N, CT, true><<<grid, 256, lds, a.stream>>>(a, waves);
    } else {
        const size_t lds = CF::walk_bytes(sw, CF::NT, 2);
        if (!lds_limit(k_delta_rev<T, N, CT>, lds)) return 7;
        k_delta_rev<T, N, CT><<<grid, 256, lds, a.stream>>>(a, waves);
    }
    return hipGetLastError() == hipSuccess ? 0 : 7;
}

template <typename T, int N>
int walk_n(const Args& a, const Slice& s, int which) {
    if constexpr (std::is_same<T, bf16>::value && N <= 128) {
        if (s.ct == 2) return walk<T, N, 2>(a, s.waves, which);
    }
    return walk<T, N, 1>(a, s.waves, which);
}

// Whether the walks run on tables stored as fragments (k_delta_dma, k_delta_team, k_delta_adj).
inline bool dma_walk(bool bf16_dtype, int64_t N) { return bf16_dtype && N >= 64; }

// Heads of a group that one wave of the preparation takes, sharing their K K^T and Q K^T: up
// to 4 while that leaves 8 waves per SIMD.
inline int prep_heads(int64_t ntab, int64_t H, int64_t G) {
    int s = 4;
    while (s > 1 && (s > H / G || ntab * G * ((H / G + s - 1) / s) < 8192)) s >>= 1;
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
// fragments are then read once for both; at dstate 256 LDS leaves no room).
inline int team_tiles(int64_t bh, int64_t P, int64_t N) { return N <= 128 && P >= 32 && bh * P > 256 * 16 ? 2 : 1; }
template <int N, int CT, bool SAVE>
int walk_team(const Args& a) {
    const unsigned grid = (unsigned)((int64_t)a.rows.nrows * a.H * (a.P / (16 * CT)));
    // (at dstate 256 the backward's tables leave room for one K buffer only)
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
// Teams while each has a CU of its own, and at any number of chains where a head is too narrow for
// a work-group of four waves to share its tables; else a wave per 16 columns.  Forward of 2048
// tokens, whole call (us, team / wave; M then in one term): headdim 64, dstate 128: 32 heads
// 67 / 127, 128 heads 121 / 153, 192 heads 213 / 172, 768 heads 657 / 493; headdim 64, dstate 256:
// 64 heads 114 / 201, 96 heads 202 / 216, 192 heads 313 / 254; headdim 32, dstate 128: 256 heads
// 154 / 182, 768 heads 418 / 406; headdim 32, dstate 256: 256 heads 259 / 271, 768 heads 670 / 719;
// headdim 16, 768 heads: dstate 128 342 / 347, dstate 256 440 / 800.
inline bool team_walk(int64_t bh, int64_t P, int64_t N) {
    return P < (N <= 128 ? 32 : 64) || bh * P <= 256 * 16 * (N <= 128 ? 2 : 1);
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
        const Slice s = slice_of(std::is_same<T, bf16>::value, (int64_t)a.rows.nrows * a.H, a.P, N);
        prep<T, N, kPlain>(a);
        return walk_n<T, N>(a, s, 0);
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
        const Slice s = slice_of(std::is_same<T, bf16>::value, (int64_t)a.rows.nrows * a.H, a.P, N);
        prep<T, N, kPlain>(a);
        st = walk_n<T, N>(a, s, 1);
        if (!st) st = walk_n<T, N>(a, s, 2);
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
