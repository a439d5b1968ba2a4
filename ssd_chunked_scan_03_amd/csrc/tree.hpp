// tree.hpp -- a tree of drafted tokens over held states.  With E_k and W_kj the decays to node k
// along its path from the held state h and from node j (1 for j = k, 0 where j is not on the path):
//
//   M_kj = W_kj (C_k . B_j),   T_kj = beta_k W_kj (B_k . B_j) (j != k)
//   scan:   y = diag(E) C h^T + M x + D x
//   delta:  (I + T) u = beta (x - diag(E) B h^T),   y = diag(E) C h^T + M u
//
// A parent precedes its node, so T is strictly lower and I + T is solved tile by tile:
// u_t = (I + T_tt)^-1 (r_t - T_{t,<t} u_{<t}) for tiles t of 16 nodes.  The state is read once and no
// state is formed per node.
//
// One work-group per (row, head, up to 64 columns of headdim), a wave per 16 columns.  The waves share
// the forming of M and T (a node tile each, B B^T and B C^T on the matrix cores, weighted by the
// decays) through LDS; every other product stays in its wave: the state's rows are operand fragments
// straight from memory, and accumulators (rows 4 (l / 16) + e of a node tile, column l % 16) feed the
// next product as operands whose k index runs 16 (e / 4) + 4 (l / 16) + e % 4.  Nodes are taken 64 at a
// time, against panels of 64 nodes up to their own.
//
// Precision.  bfloat16 problems: float32 factors (state, M, T, inverse, right side, u) enter the matrix
// cores as two bfloat16 terms, which leaves 2^-16 of them, far below y's own rounding; float32 problems
// run on the float32 matrix cores.  Decay sums are formed along each path in float64: the difference
// of two running sums would lose what a strong decay above leaves of a weak one.
#pragma once

#include "delta_launch.hpp"
#include "pool.hpp"

namespace ssd {
namespace pool {

using delta::Sp;
using delta::join;

constexpr int kPanel = 64;

template <typename T> constexpr int kTwo = std::is_same<T, bf16>::value ? 2 : 1;

// c += a b: both in two terms (their smallest product left out), or b exact
template <typename T> struct Op { typename V8<T>::type t[kTwo<T>]; };
__device__ __forceinline__ f32x4 mul(f32x4 c, const Op<bf16>& a, const Op<bf16>& b) {
    c = mma(c, a.t[1], b.t[0]);
    c = mma(c, a.t[0], b.t[1]);
    return mma(c, a.t[0], b.t[0]);
}
__device__ __forceinline__ f32x4 mul(f32x4 c, const Op<float>& a, const Op<float>& b) { return mma(c, a.t[0], b.t[0]); }
__device__ __forceinline__ f32x4 mul(f32x4 c, const Op<bf16>& a, bf16x8 b) { return mma(mma(c, a.t[1], b), a.t[0], b); }
__device__ __forceinline__ f32x4 mul(f32x4 c, const Op<float>& a, f32x8 b) { return mma(c, a.t[0], b); }
__device__ __forceinline__ f32x4 mul(f32x4 c, bf16x8 a, const Op<bf16>& b) { return mma(mma(c, a, b.t[1]), a, b.t[0]); }
__device__ __forceinline__ f32x4 mul(f32x4 c, f32x8 a, const Op<float>& b) { return mma(c, a, b.t[0]); }

__device__ __forceinline__ void split(f32x8 v, Op<bf16>& o) {
    Sp<bf16> s;
    delta::split8<2>(v, s);
    o.t[0] = s.t[0];
    o.t[1] = s.t[1];
}
__device__ __forceinline__ void split(f32x8 v, Op<float>& o) { o.t[0] = v; }

// Tables of operand fragments in LDS, [fragment][term][lane][8]; v is one half of a lane's fragment.
__device__ __forceinline__ void put(bf16* tab, int f, int half, int lane, f32x4 v) {
    bf16x4 o[2];
    delta::split4<2>(v, o);
    st4(tab + ((f * 2 + 0) * 64 + lane) * 8 + 4 * half, o[0]);
    st4(tab + ((f * 2 + 1) * 64 + lane) * 8 + 4 * half, o[1]);
}
__device__ __forceinline__ void put(float* tab, int f, int half, int lane, f32x4 v) { st4(tab + (f * 64 + lane) * 8 + 4 * half, v); }
template <typename T>
__device__ __forceinline__ Op<T> get(const T* tab, int f, int lane) {
    Op<T> o;
#pragma unroll
    for (int t = 0; t < kTwo<T>; ++t) o.t[t] = ld8(tab + ((f * kTwo<T> + t) * 64 + lane) * 8);
    return o;
}
// The inverse of a diagonal tile, [lane]: its terms side by side (one product takes both), or alone.
__device__ __forceinline__ void put_inv(bf16* tab, int lane, f32x4 v) {
    bf16x4 o[2];
    delta::split4<2>(v, o);
    st8(tab + lane * 8, join(o[0], o[1]));
}
__device__ __forceinline__ void put_inv(float* tab, int lane, f32x4 v) { st4(tab + lane * 4, v); }
__device__ __forceinline__ f32x4 times_inv(const bf16* tab, int lane, f32x4 v) {
    bf16x4 o[2];
    delta::split4<2>(v, o);
    const bf16x8 a = ld8(tab + lane * 8);
    const bf16x4 zero = {};
    return mma(mma(f32x4{0.f, 0.f, 0.f, 0.f}, a, join(o[1], zero)), a, join(o[0], o[0]));
}
__device__ __forceinline__ f32x4 times_inv(const float* tab, int lane, f32x4 v) {
    return delta::mma16(f32x4{0.f, 0.f, 0.f, 0.f}, ld4(tab + lane * 4), v);
}

struct Node {
    double s;    // binary orders of decay of its step
    int par;
    float beta;  // NaN: the delta rule cannot use the node, nor what is below it
};

constexpr int kTableBytes = 4096;  // of a node tile's M (or T) against a panel
// LDS of a work-group: nodes, decays from the held state, bad columns, tables, and the u of earlier panels.
struct TreeLds {
    int nodes, decay, badx, m, t, inv, u, total;
    __host__ __device__ TreeLds(int K, int waves, bool rule_delta) {
        const bool one = K <= kPanel;
        const int kp = (K + kPanel - 1) / kPanel * kPanel, panels = kp / kPanel;
        // (a tile's own panel has no tiles behind its own: half the table for the first two of four)
        const int tab = one ? 3 * kTableBytes : 4 * kTableBytes;
        m = 0;
        t = m + tab;
        inv = t + (rule_delta ? tab : 0);
        nodes = inv + (rule_delta ? 4 * 1024 : 0);
        decay = nodes + kp * (int)sizeof(Node);
        badx = decay + kp * 4;
        u = badx + panels * waves * 16 * 8;
        total = u + (rule_delta ? (panels - 1) * waves * kTableBytes : 0);
    }
    // Tile kt's table: whole panels 4 KiB a tile, single panels 2, 2, 4, 4.
    static __device__ int at(int kt, bool one) { return one ? (kt < 2 ? kt * 2048 : (kt - 1) * kTableBytes) : kt * kTableBytes; }
};

__device__ __forceinline__ bool odd_bits(float v) { return (__builtin_bit_cast(unsigned, v) & 0x7f800000u) == 0x7f800000u; }
__device__ __forceinline__ bool any_odd(bf16x8 v) {
    const u32x4v w = __builtin_bit_cast(u32x4v, v);
    bool o = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) o |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
    return o;
}
__device__ __forceinline__ bool any_odd(f32x8 v) {
    bool o = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) o |= odd_bits(v[e]);
    return o;
}
// orders LDS traffic of one wave's lanes (LDS serves a wave in order; this keeps the compiler to it)
__device__ __forceinline__ void wave_sync() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// Accumulators that a branch ends on: the compiler may let the code behind the branch read them before the
// matrix instruction has written them (seen: a read one instruction later, where eight have to lie between),
// so the wait is stated here.
__device__ __forceinline__ void settle(f32x4& v) { asm volatile("s_nop 7\n\ts_nop 3" : "+v"(v)); }

// (I + t)^-1 of a strictly lower 16 x 16 tile: lane (q, k) holds t[k][4 q + e] and gets the inverse's.
// Row by row: X_k = e_k - sum_{j < k} t_kj X_j, row j of X from its lanes to all by DPP.
template <int J>
__device__ __forceinline__ void inv_step(f32x4& x, const float (&row)[16]) {
    if constexpr (J < 15) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] -= row[J] * delta::lane_turn<0x150 + J>((float)x[e]);
        inv_step<J + 1>(x, row);
    }
}
__device__ __forceinline__ f32x4 inverse16(f32x4 t, float* scratch, int lane) {
    const int k = lane & 15, q = lane >> 4;
    st4(scratch + k * 16 + 4 * (q ^ (k & 3)), t);
    wave_sync();
    float row[16];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const f32x4 v = ld4(scratch + k * 16 + 4 * (c ^ (k & 3)));
#pragma unroll
        for (int e = 0; e < 4; ++e) row[4 * c + e] = v[e];
    }
    wave_sync();
    f32x4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = 4 * q + e == k ? 1.f : 0.f;
    inv_step<0>(x, row);
    return x;
}

// 16 x 4 values of a node tile as its accumulators hold them (lane: nodes 4 q + e, column l % 16) from
// and to memory.  bfloat16 moves 8 bytes a lane through a transpose in the ALU.
__device__ __forceinline__ f32x4 load_x(const bf16* x, int64_t xs, int k0, int K, int lane, unsigned sel, bool upper) {
    const int k = k0 + 4 * (lane >> 4) + (lane & 3);
    delta::u32x2v v = {0, 0};
    if (k < K) v = *reinterpret_cast<const delta::u32x2v*>(x + (int64_t)k * xs + 4 * ((lane & 15) >> 2));
    return delta::floats(delta::quad_t(v, sel, upper));
}
__device__ __forceinline__ f32x4 load_x(const float* x, int64_t xs, int k0, int K, int lane, unsigned, bool) {
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int k = k0 + 4 * (lane >> 4) + e;
        v[e] = k < K ? x[(int64_t)k * xs + (lane & 15)] : 0.f;
    }
    return v;
}
__device__ __forceinline__ void store_y(bf16* y, int64_t ys, int k0, int K, int lane, unsigned sel, bool upper, f32x4 v) {
    const delta::u32x2v w = delta::quad_t(delta::u32x2v{delta::cvt2(v[0], v[1]), delta::cvt2(v[2], v[3])}, sel, upper);
    const int k = k0 + 4 * (lane >> 4) + (lane & 3);
    if (k < K) *reinterpret_cast<delta::u32x2v*>(y + (int64_t)k * ys + 4 * ((lane & 15) >> 2)) = w;
}
__device__ __forceinline__ void store_y(float* y, int64_t ys, int k0, int K, int lane, unsigned, bool, f32x4 v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int k = k0 + 4 * (lane >> 4) + e;
        if (k < K) y[(int64_t)k * ys + (lane & 15)] = v[e];
    }
}
__device__ __forceinline__ bf16x8 pair8(const bf16*, f32x4 a, f32x4 b) {  // exact: both are bfloat16 already
    typedef delta::u32x2v U2;
    return __builtin_bit_cast(bf16x8, u32x4v{delta::cvt2(a[0], a[1]), delta::cvt2(a[2], a[3]), delta::cvt2(b[0], b[1]),
                                             delta::cvt2(b[2], b[3])});
}
__device__ __forceinline__ f32x8 pair8(const float*, f32x4 a, f32x4 b) { return join(a, b); }

template <typename T, int N, bool DELTA>
__global__ __launch_bounds__(256) void k_tree(Args a) {
    typedef typename V8<T>::type F8;
    constexpr int KS = N < 32 ? 1 : N / 32;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int waves = blockDim.x >> 6, K = (int)a.T, P = a.P, H = a.H;
    const int slabs = P / (16 * waves);
    const int64_t bh = blockIdx.x / slabs;
    const int slab = blockIdx.x % slabs, h = (int)(bh % H), g = h / (H / a.G);
    const int64_t bi = bh / H, row0 = bi * K;
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), l16 = lane & 15, q = lane >> 4;
    const int p0 = (slab * waves + w) * 16;
    const unsigned sel = delta::quad_sel(lane);
    const bool upper = (lane & 2) != 0, one = K <= kPanel;
    const TreeLds at(K, waves, DELTA);
    Node* nodes = reinterpret_cast<Node*>(smem + at.nodes);
    float* decay = reinterpret_cast<float*>(smem + at.decay);  // E; -1 absent, -2 not computable
    unsigned long long* badx = reinterpret_cast<unsigned long long*>(smem + at.badx);
    const T* x = static_cast<const T*>(a.x) + row0 * a.xs + h * P + p0;
    const T* Bm = static_cast<const T*>(a.B) + row0 * a.bs + g * N;
    const T* Cm = static_cast<const T*>(a.C) + row0 * a.cs + g * N;
    T* y = static_cast<T*>(a.y) + (row0 * H + h) * P + p0;
    const int64_t ys = (int64_t)H * P;
    const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
    const int slot = a.slots[bi];
    if (slot < 0 || slot >= a.S) {
        for (int k0 = 0; k0 < K; k0 += 16) store_y(y, ys, k0, K, lane, sel, upper, zero4);
        return;
    }

    // the state's rows as operands: lane (q, l16) holds row p0 + l16, elements 32 ks + 8 q .. + 7
    f32x8 hf[KS];
    const bool has = N >= 32 || q < 2;  // (dstate 16 fills half a fragment)
    {
        const float* hp = a.pool + slot * a.ss + (int64_t)(h * P + p0 + l16) * N + 8 * (N >= 32 ? q : q & 1);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) hf[ks] = ld8(hp + 32 * ks);
    }
    // row `node` (clamped: rows past the last are never used) of B or C
    auto frag = [&](const T* m, int64_t stride, int node, int ks) {
        const F8 v = ld8(m + (int64_t)(node < K ? node : K - 1) * stride + 32 * ks + 8 * (N >= 32 ? q : q & 1));
        return N >= 32 ? v : sel8(has, v);
    };

    const double Ah = (double)a.A[h] * 1.4426950408889634;
    if (DELTA) {
        // N / 8 lanes a node: its row of B as well
        constexpr int R = N / 8;
        const T* beta = static_cast<const T*>(a.beta);
        for (int k0 = 0; k0 < K; k0 += (int)blockDim.x / R) {
            const int k = k0 + tid / R;
            const bool in = k < K;
            const bool odd = in && any_odd(ld8(Bm + (int64_t)(in ? k : 0) * a.bs + 8 * (tid % R)));
            const unsigned long long who = __ballot(odd) >> (lane / R * R);
            if (in && tid % R == 0) {
                Node n;
                n.s = (double)a.dt[(row0 + k) * H + h] * Ah;
                n.par = a.parents[row0 + k];
                n.beta = to_f(beta[(row0 + k) * H + h]);
                const bool bad = (who & ((1ull << R) - 1)) != 0 || !(n.s < __builtin_huge_val()) || odd_bits(n.beta);
                if (bad) n.beta = __builtin_nanf("");
                nodes[k] = n;
            }
        }
    } else {
        for (int k = tid; k < K; k += blockDim.x) {
            Node n;
            n.s = (double)a.dt[(row0 + k) * H + h] * Ah;
            n.par = a.parents[row0 + k];
            n.beta = 0.f;
            nodes[k] = n;
        }
    }
    const int panels = (K + kPanel - 1) / kPanel;
    for (int i = lane; i < 16 * panels; i += 64) badx[((i >> 4) * waves + w) * 16 + (i & 15)] = 0;
    __syncthreads();

    bool anybad = false;
    // x of a panel's tile, as accumulators: absent nodes and bad values are zero (bad ones noted)
    auto take_x = [&](int k0) {
        f32x4 v = load_x(x, a.xs, k0, K, lane, sel, upper);
        if (k0 >= K) return v;
        const f32x4 e4 = ld4(decay + k0 + 4 * q);
        unsigned odd = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool there = !(e4[e] < 0.f) && k0 + 4 * q + e < K;
            if (there && odd_bits(v[e])) odd |= 1u << e;
            v[e] = there && !odd_bits(v[e]) ? v[e] : 0.f;
        }
        if (__ballot(odd != 0)) {
            anybad = true;
            if (odd) atomicOr(&badx[((k0 >> 6) * waves + w) * 16 + l16], (unsigned long long)odd << ((k0 & 63) + 4 * q));
            wave_sync();
        }
        return v;
    };

    Op<T> hs[KS];
    for (int s = 0; s < panels; ++s) {
        const int q0 = s * kPanel, nk = (K - q0 + 15) / 16 < 4 ? (K - q0 + 15) / 16 : 4;
        f32x4 O[4], R[4], xt[4];
        for (int sp = 0; sp <= s; ++sp) {
            const bool own = sp == s;
            const int j0 = sp * kPanel;
            if (s > 0) __syncthreads();  // the tables are free
            // ---- tables of node tile kt against panel sp ----
            for (int kt = w; kt < nk; kt += waves) {
                T* mt = reinterpret_cast<T*>(smem + at.m + TreeLds::at(kt, one));
                T* tt = reinterpret_cast<T*>(smem + at.t + TreeLds::at(kt, one));
                float* wt = reinterpret_cast<float*>(mt);  // decays first, in M's place
                const int wide = one && kt < 2 ? 32 : 64, gm = wide / 4 - 1, k = q0 + 16 * kt + l16;
                for (int i = lane * 4; i < 16 * wide; i += 256) st4(wt + i, f32x4{-1.f, -1.f, -1.f, -1.f});
                wave_sync();
                bool ok = k < K, bad = false;
                float bk = 0.f;
                double sum = 0.0;
                if (ok) {
                    int j = k;
                    Node n = nodes[j];
                    bk = n.beta;
                    for (;;) {
                        const int c = j - j0;
                        if (c >= 0 && c < kPanel && ((j >> 2) & 3) == q)
                            wt[l16 * wide + ((c >> 2 ^ (l16 & gm)) << 2) + (c & 3)] = exp2f_fast((float)sum);
                        sum += n.s;
                        if (DELTA) bad |= n.beta != n.beta;
                        ok = n.par >= -1 && n.par < j;
                        if (!ok || n.par < 0) break;
                        j = n.par;
                        n = nodes[j];
                    }
                }
                if (sp == 0 && q == 0) decay[k] = !ok ? -1.f : bad ? -2.f : exp2f_fast((float)sum);
                wave_sync();
                const int jn = own ? kt + 1 : 4;
                f32x4 w4[4];
#pragma unroll
                for (int jt = 0; jt < 4; ++jt)
                    if (jt < jn) {
                        w4[jt] = ld4(wt + l16 * wide + ((4 * jt + q) ^ (l16 & gm)) * 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) w4[jt][e] = ok && !bad ? w4[jt][e] : -1.f;
                    }
                wave_sync();
                F8 cf[KS], bf[KS];
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    cf[ks] = frag(Cm, a.cs, k, ks);
                    if (DELTA) bf[ks] = frag(Bm, a.bs, k, ks);
                }
                f32x4 diag = zero4;
#pragma unroll
                for (int jt = 0; jt < 4; ++jt)
                    if (jt < ((jn + 1) & ~1)) {
                        f32x4 m = zero4, t = zero4;
                        if (jt < jn) {
                            f32x4 gc = zero4, gb = zero4;
#pragma unroll
                            for (int ks = 0; ks < KS; ++ks) {
                                const F8 bj = frag(Bm, a.bs, j0 + 16 * jt + l16, ks);
                                gc = mma(gc, bj, cf[ks]);
                                if (DELTA) gb = mma(gb, bj, bf[ks]);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const bool off = w4[jt][e] < 0.f;
                                m[e] = off ? 0.f : w4[jt][e] * gc[e];
                                if (DELTA) t[e] = off || j0 + 16 * jt + 4 * q + e == k ? 0.f : bk * w4[jt][e] * gb[e];
                            }
                        }
                        put(mt, jt >> 1, jt & 1, lane, m);
                        if (DELTA) {
                            if (own && jt == kt) {
                                diag = t;
                                t = zero4;
                            }
                            put(tt, jt >> 1, jt & 1, lane, t);
                        }
                    }
                if (DELTA && own) {
                    T* inv = reinterpret_cast<T*>(smem + at.inv + kt * 1024);
                    put_inv(inv, lane, inverse16(diag, reinterpret_cast<float*>(inv), lane));
                }
            }
            __syncthreads();
            if (sp == 0) {
                // ---- what the held state gives: O = diag(E) C h^T, R = -beta diag(E) B h^T ----
                if (s == 0) {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        if (N < 32) hf[ks] = sel8(has, hf[ks]);
                        split(hf[ks], hs[ks]);
                    }
                }
#pragma unroll
                for (int kt = 0; kt < 4; ++kt)
                    if (kt < nk) {
                        const int k = q0 + 16 * kt;
                        f32x4 o = zero4, v = zero4;
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) {
                            o = mul(o, frag(Cm, a.cs, k + l16, ks), hs[ks]);
                            if (DELTA) v = mul(v, frag(Bm, a.bs, k + l16, ks), hs[ks]);
                        }
                        const f32x4 e4 = ld4(decay + k + 4 * q);
                        xt[kt] = take_x(k);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            O[kt][e] = e4[e] * o[e];
                            if (DELTA) {
                                const int n = k + 4 * q + e;
                                R[kt][e] = e4[e] < 0.f || n >= K ? 0.f : nodes[n].beta * (xt[kt][e] - e4[e] * v[e]);
                            }
                        }
                    }
            }
            // ---- panel sp's part of R and O ----
            if constexpr (!DELTA) {
                F8 xf[2];
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    f32x4 lo = zero4, hi = zero4;
                    if (own) {
                        if (2 * f < nk) lo = xt[2 * f];
                        if (2 * f + 1 < nk) hi = xt[2 * f + 1];
                    } else {
                        lo = take_x(j0 + 32 * f);
                        hi = take_x(j0 + 32 * f + 16);
                    }
                    xf[f] = pair8(x, lo, hi);
                }
#pragma unroll
                for (int kt = 0; kt < 4; ++kt)
                    if (kt < nk) {
                        const T* mt = reinterpret_cast<const T*>(smem + at.m + TreeLds::at(kt, one));
#pragma unroll
                        for (int f = 0; f < 2; ++f)
                            if (!own || 2 * f <= kt) O[kt] = mul(O[kt], get(mt, f, lane), xf[f]);
                        settle(O[kt]);
                    }
            } else {
                Op<T> uf[2];
                T* us = reinterpret_cast<T*>(smem + at.u + (sp * waves + w) * kTableBytes);
                if (own) {
                    f32x4 u[4] = {zero4, zero4, zero4, zero4};
                    split(join(zero4, zero4), uf[0]);
                    split(join(zero4, zero4), uf[1]);
#pragma unroll
                    for (int kt = 0; kt < 4; ++kt)
                        if (kt < nk) {
                            const T* tt = reinterpret_cast<const T*>(smem + at.t + TreeLds::at(kt, one));
                            f32x4 t = zero4;
#pragma unroll
                            for (int f = 0; f < 2; ++f)
                                if (2 * f < kt) t = mul(t, get(tt, f, lane), uf[f]);
                            u[kt] = times_inv(reinterpret_cast<const T*>(smem + at.inv + kt * 1024), lane, R[kt] - t);
                            split(join(u[kt & ~1], u[kt | 1]), uf[kt >> 1]);
                        }
                    if (s + 1 < panels) {
#pragma unroll
                        for (int f = 0; f < 2; ++f)
#pragma unroll
                            for (int t = 0; t < kTwo<T>; ++t) st8(us + ((f * kTwo<T> + t) * 64 + lane) * 8, uf[f].t[t]);
                    }
                } else {
                    uf[0] = get(us, 0, lane);
                    uf[1] = get(us, 1, lane);
                }
                if (!own) {
#pragma unroll
                    for (int kt = 0; kt < 4; ++kt)
                        if (kt < nk) {
                            const T* tt = reinterpret_cast<const T*>(smem + at.t + TreeLds::at(kt, one));
                            f32x4 t = mul(mul(zero4, get(tt, 0, lane), uf[0]), get(tt, 1, lane), uf[1]);
                            settle(t);
                            R[kt] -= t;
                        }
                }
#pragma unroll
                for (int kt = 0; kt < 4; ++kt)
                    if (kt < nk) {
                        const T* mt = reinterpret_cast<const T*>(smem + at.m + TreeLds::at(kt, one));
#pragma unroll
                        for (int f = 0; f < 2; ++f)
                            if (!own || 2 * f <= kt) O[kt] = mul(O[kt], get(mt, f, lane), uf[f]);
                        settle(O[kt]);
                    }
            }
        }
        // ---- y ----
        const float D = a.D ? a.D[h] : 0.f;
        const float nan = __builtin_nanf("");
#pragma unroll
        for (int kt = 0; kt < 4; ++kt)
            if (kt < nk) {
                const int k0 = q0 + 16 * kt;
                const f32x4 e4 = ld4(decay + k0 + 4 * q);
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float o = DELTA ? O[kt][e] : O[kt][e] + D * xt[kt][e];
                    v[e] = e4[e] == -1.f ? 0.f : e4[e] == -2.f ? nan : o;
                    if (anybad && k0 + 4 * q + e < K && !(e4[e] < 0.f)) {
                        // a bad x on the node's path
                        bool hit = false;
                        for (int j = k0 + 4 * q + e; j >= 0; j = nodes[j].par)
                            hit |= badx[((j >> 6) * waves + w) * 16 + l16] >> (j & 63) & 1;
                        if (hit) v[e] = nan;
                    }
                }
                store_y(y, ys, k0, K, lane, sel, upper, v);
            }
    }
}

template <typename T, int N>
int run_tree_n(const Args& a) {
    const int waves = a.P < 64 ? a.P / 16 : 4;
    const size_t lds = (size_t)TreeLds((int)a.T, waves, a.beta != nullptr).total;
    auto kernel = a.beta ? k_tree<T, N, true> : k_tree<T, N, false>;
    if (!delta::lds_limit(kernel, lds)) return 7;
    kernel<<<(unsigned)(a.b * a.H * (a.P / (16 * waves))), 64 * waves, lds, a.stream>>>(a);
    return hipGetLastError() == hipSuccess ? 0 : 7;
}
template <typename T>
int run_tree(const Args& a) {
    switch (a.N) {
        case 16: return run_tree_n<T, 16>(a);
        case 32: return run_tree_n<T, 32>(a);
        case 64: return run_tree_n<T, 64>(a);
        case 128: return run_tree_n<T, 128>(a);
        case 256: return run_tree_n<T, 256>(a);
        default: return 3;
    }
}

int tree_bf16(const Args& a);
int tree_f32(const Args& a);

}  // namespace pool
}  // namespace ssd
