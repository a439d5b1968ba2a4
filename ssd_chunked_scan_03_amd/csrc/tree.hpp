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

// LDS of a work-group.  kp: nodes rounded up to panels; hb: heads that it takes one after another.
constexpr int kTableBytes = 4096;  // of a node tile's M (or T) against a panel
struct TreeLds {
    int m, t, inv, gc, gb, mask, c, e, beta, ptr, badx, u, total;
    __host__ __device__ TreeLds(int K, int waves, int hb, bool rule_delta) {
        const bool one = K <= kPanel;
        const int kp = (K + kPanel - 1) / kPanel * kPanel, panels = kp / kPanel;
        // (a tile's own panel has no tiles behind its own: half the table for the first two of four)
        const int tab = one ? 3 * kTableBytes : 4 * kTableBytes, g = one ? 10 * 1024 : 0;
        m = 0;                                              // [tile] M as fragments
        t = m + tab;                                        // [tile] T
        inv = t + (rule_delta ? tab : 0);                   // [tile] the diagonal tiles' inverses
        gc = inv + (rule_delta ? 4 * 1024 : 0);             // [tile pair] B C^T, one panel
        gb = gc + g;                                        // [tile pair] B B^T
        mask = gb + (rule_delta ? g : 0);                   // [node][panel] the node and those above it
        c = mask + kp * panels * 8;                         // [head][node] binary orders of decay from the held state
        e = c + hb * kp * 8;                                // [head][node] E; -1 absent, -2 not computable
        beta = e + hb * kp * 4;                             // [head][node]
        ptr = beta + (rule_delta ? hb * kp * 4 : 0);        // [node] while the paths are formed
        badx = ptr + (one ? 64 : kp * 4);                   // [panel][column] nodes whose x is not finite
        u = badx + (one ? 0 : panels * waves * 16 * 8);     // [panel][wave] u of the panels before the last
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

// A step's binary orders of decay, kept to where sums of 256 of them and differences of those are exact
// enough in float64 (2^20 is far past what any float32 exponential tells from 0): a decay to nothing
// above a node takes nothing from what the nodes below it tell apart.
__device__ __forceinline__ double orders(float dt, double A) {
    const double s = (double)dt * A;
    return s < -1048576.0 ? -1048576.0 : s > 1048576.0 ? 1048576.0 : s;  // (a NaN stays)
}

template <typename T, int N, bool DELTA, bool ONE>
__global__ __launch_bounds__(256) void k_tree(Args a, int hb) {
    typedef typename V8<T>::type F8;
    typedef unsigned long long u64;
    constexpr int KS = N < 32 ? 1 : N / 32;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int waves = blockDim.x >> 6, K = (int)a.T, P = a.P, H = a.H, hg = H / a.G;
    const int slabs = P / (16 * waves), chunks = (hg + hb - 1) / hb;
    // blocks k, k + 8, ... run on one XCD: each takes a contiguous range, so that a row's B, C and dt stay in its L2
    const int nb = gridDim.x;
    int64_t id = nb % 8 == 0 ? (int64_t)(blockIdx.x % 8) * (nb / 8) + blockIdx.x / 8 : blockIdx.x;
    const int slab = (int)(id % slabs);
    id /= slabs;
    const int chunk = (int)(id % chunks);
    id /= chunks;
    const int g = (int)(id % a.G);
    const int64_t bi = id / a.G, row0 = bi * K;
    const int h0 = g * hg + chunk * hb, nh = hg - chunk * hb < hb ? hg - chunk * hb : hb;
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), l16 = lane & 15, q = lane >> 4;
    const int p0 = (slab * waves + w) * 16;
    const unsigned sel = delta::quad_sel(lane);
    const bool upper = (lane & 2) != 0;
    const int kp = ONE ? kPanel : (K + kPanel - 1) / kPanel * kPanel, panels = kp / kPanel;
    const TreeLds at(ONE ? kPanel : K, waves, hb, DELTA);
    u64* mask = reinterpret_cast<u64*>(smem + at.mask);
    double* cs = reinterpret_cast<double*>(smem + at.c);
    float* decay = reinterpret_cast<float*>(smem + at.e);
    float* betas = reinterpret_cast<float*>(smem + at.beta);
    const T* Bm = static_cast<const T*>(a.B) + row0 * a.bs + g * N;
    const T* Cm = static_cast<const T*>(a.C) + row0 * a.cs + g * N;
    const int64_t ys = (int64_t)H * P;
    const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
    const int slot = a.slots[bi];
    if (slot < 0 || slot >= a.S) {
        for (int hh = 0; hh < nh; ++hh)
            for (int k0 = 0; k0 < K; k0 += 16)
                store_y(static_cast<T*>(a.y) + (row0 * H + h0 + hh) * P + p0, ys, k0, K, lane, sel, upper, zero4);
        return;
    }
    const bool has = N >= 32 || q < 2;  // (dstate 16 fills half a fragment)
    const int n0 = 8 * (N >= 32 ? q : q & 1);
    // the state's rows as operands: lane (q, l16) holds row p0 + l16, elements 32 ks + 8 q .. + 7
    f32x8 hf[KS];
    auto load_state = [&](int h) {
        const float* hp = a.pool + slot * a.ss + (int64_t)(h * P + p0 + l16) * N + n0;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) hf[ks] = ld8(hp + 32 * ks);
    };
    // row `node` (clamped: rows past the last are never used) of B or C
    auto frag = [&](const T* m, int64_t stride, int node, int ks) {
        const F8 v = ld8(m + (int64_t)(node < K ? node : K - 1) * stride + 32 * ks + n0);
        return N >= 32 ? v : sel8(has, v);
    };
    const T* beta = static_cast<const T*>(a.beta);

    // ---- what the heads share, and every head's decays ----
    if constexpr (ONE) {
        const int k = lane;
        const int par = k < K ? a.parents[row0 + k] : -2;
        load_state(h0);
        float* gc = reinterpret_cast<float*>(smem + at.gc);
        float* gb = reinterpret_cast<float*>(smem + at.gb);
        u64* badb = reinterpret_cast<u64*>(smem + at.ptr);  // [tile] nodes whose row of B is not finite
        for (int kt = w; 16 * kt < K; kt += waves) {
            F8 cf[KS], bf[KS];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                cf[ks] = frag(Cm, a.cs, 16 * kt + l16, ks);
                bf[ks] = frag(Bm, a.bs, 16 * kt + l16, ks);
            }
            for (int jt = 0; jt <= kt; ++jt) {
                f32x4 c = zero4, b = zero4;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const F8 bj = jt == kt ? bf[ks] : frag(Bm, a.bs, 16 * jt + l16, ks);
                    c = mma(c, bj, cf[ks]);
                    if (DELTA) b = mma(b, bj, bf[ks]);
                }
                settle(c);
                const int tile = (kt * (kt + 1) / 2 + jt) * 256 + lane * 4;
                st4(gc + tile, c);
                if (DELTA) {
                    settle(b);
                    st4(gb + tile, b);
                    if (jt == kt) {
                        // |B_k|^2 on the diagonal tells whether the row is finite
                        const float d = l16 & 2 ? (l16 & 1 ? b[3] : b[2]) : (l16 & 1 ? b[1] : b[0]);
                        u64 who = __ballot(q == l16 >> 2 && odd_bits(d));
                        who |= who >> 32;
                        if (lane == 0) badb[kt] = ((who | who >> 16) & 0xffff) << (16 * kt);
                    }
                }
            }
        }
        // the paths, by doubling: pr[r] is the node 2^r above
        bool there = k < K && par >= -1 && par < k;
        u64 mk = 1ull << k;
        int pr[6], p = there && par >= 0 ? par : -1, rounds = 0;
#pragma unroll
        for (int r = 0; r < 6; ++r) {
            pr[r] = p;
            if (rounds == r && __ballot(p >= 0)) {
                const int from = p < 0 ? lane : p;
                mk |= __shfl(mk, from, 64);
                const int ok = __shfl((int)there, from, 64), up = __shfl(p, from, 64);
                there = there && ok;
                p = p < 0 ? -1 : up;
                rounds = r + 1;
            }
        }
        if (w == 0) mask[k] = mk;
        if (DELTA) __syncthreads();
        for (int hh = w; hh < nh; hh += waves) {
            const int64_t at_k = (row0 + (k < K ? k : K - 1)) * H + h0 + hh;
            double c = orders(a.dt[at_k], (double)a.A[h0 + hh] * 1.4426950408889634);
            bool bad = false;
            if (DELTA) {
                const float bt = to_f(beta[at_k]);
                u64 odd = __ballot(c != c || odd_bits(bt));
                for (int kt = 0; 16 * kt < K; ++kt) odd |= badb[kt];
                bad = (mk & odd) != 0;
                betas[hh * 64 + k] = bt;
            }
#pragma unroll
            for (int r = 0; r < 6; ++r)
                if (r < rounds) {
                    const double up = __shfl(c, pr[r] < 0 ? lane : pr[r], 64);
                    if (pr[r] >= 0) c += up;
                }
            cs[hh * 64 + k] = c;
            decay[hh * 64 + k] = !there ? -1.f : bad ? -2.f : exp2f_fast((float)c);
        }
    } else {
        load_state(h0);
        constexpr int R = N / 8;
        int* ptr = reinterpret_cast<int*>(smem + at.ptr);
        u64* badx = reinterpret_cast<u64*>(smem + at.badx);
        const double Ah = (double)a.A[h0] * 1.4426950408889634;
        for (int i = lane; i < 16 * panels; i += 64) badx[((i >> 4) * waves + w) * 16 + (i & 15)] = 0;
        // N / 8 lanes a node: for the delta rule its row of B as well
        for (int k0 = 0; k0 < kp; k0 += (int)blockDim.x / R) {
            const int k = k0 + tid / R;
            const bool in = k < K;
            const bool odd = DELTA && in && any_odd(ld8(Bm + (int64_t)(in ? k : 0) * a.bs + 8 * (tid % R)));
            const u64 who = __ballot(odd) >> (lane / R * R);
            if (k < kp && tid % R == 0) {
                const double s = orders(in ? a.dt[(row0 + k) * H + h0] : 0.f, Ah);
                const int par = in ? a.parents[row0 + k] : -2;
                const bool ok = par >= -1 && par < k;
                bool bad = false;
                if (DELTA) {
                    const float bt = in ? to_f(beta[(row0 + k) * H + h0]) : 0.f;
                    bad = (who & ((1ull << R) - 1)) != 0 || s != s || odd_bits(bt);
                    betas[k] = bt;
                }
                cs[k] = s;
                ptr[k] = ok ? par : -1;
                decay[k] = !ok ? -1.f : bad ? -2.f : 0.f;
                for (int i = 0; i < panels; ++i) mask[k * panels + i] = i == k >> 6 ? 1ull << (k & 63) : 0;
            }
        }
        __syncthreads();
        // the paths, by doubling; a node is absent below an absent one, and not computable below such a one
        for (int reach = 1; reach < K; reach *= 2) {
            double c[4];
            int up[4];
            float d[4];
            u64 m[4][4];
            // (at most four nodes a thread: 256 nodes, 64 threads)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = tid + i * (int)blockDim.x;
                if (k < kp) {
                    const int p = ptr[k], from = p < 0 ? k : p;
                    c[i] = p < 0 ? cs[k] : cs[k] + cs[from];
                    up[i] = p < 0 ? -1 : ptr[from];
                    const float mine = decay[k], theirs = decay[from];
                    d[i] = mine == -1.f || theirs == -1.f ? -1.f : mine < theirs ? mine : theirs;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < panels) m[i][j] = mask[k * panels + j] | mask[from * panels + j];
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = tid + i * (int)blockDim.x;
                if (k < kp) {
                    cs[k] = c[i];
                    ptr[k] = up[i];
                    decay[k] = d[i];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < panels) mask[k * panels + j] = m[i][j];
                }
            }
            __syncthreads();
        }
        for (int k = tid; k < kp; k += (int)blockDim.x)
            if (!(decay[k] < 0.f)) decay[k] = exp2f_fast((float)cs[k]);
    }
    __syncthreads();

    // M and T of node tile kt (nodes from k0) against the tiles [0, jn) of the panel from j0, as operand fragments;
    // for the node's own panel the inverse of its diagonal tile.  gj(jt, c, b): the lane's values of B C^T and B B^T.
    auto tables = [&](int hh, int kt, int k0, int j0, int jn, bool own, auto&& gj) {
        T* mt = reinterpret_cast<T*>(smem + at.m + TreeLds::at(kt, ONE));
        T* tt = reinterpret_cast<T*>(smem + at.t + TreeLds::at(kt, ONE));
        const int k = k0 + l16;
        const u64 mk = decay[hh * kp + k] < 0.f ? 0 : mask[k * panels + (j0 >> 6)];
        const double ck = cs[hh * kp + k];
        const float bk = DELTA ? betas[hh * kp + k] : 0.f;
        f32x4 diag = zero4;
#pragma unroll
        for (int jt = 0; jt < 4; ++jt)
            if (jt < ((jn + 1) & ~1)) {
                f32x4 m = zero4, t = zero4;
                if (jt < jn) {
                    f32x4 c = zero4, b = zero4;
                    gj(jt, c, b);
                    const unsigned bits = (unsigned)(mk >> (16 * jt + 4 * q)) & 15u;
                    const double* cj = cs + hh * kp + j0 + 16 * jt + 4 * q;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float f = exp2f_fast((float)(ck - cj[e]));
                        const bool on = bits >> e & 1;
                        m[e] = on ? f * c[e] : 0.f;
                        if (DELTA) t[e] = on && j0 + 16 * jt + 4 * q + e != k ? bk * f * b[e] : 0.f;
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
    };
    // x of a tile as accumulators, with zeros for absent nodes and for values that are not finite; the latter's
    // nodes (bits 4 q + e of the tile) come back in `odd`
    auto clean_x = [&](f32x4 v, int hh, int k0, unsigned& odd) {
        const f32x4 e4 = ld4(decay + hh * kp + k0 + 4 * q);
        odd = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool there = !(e4[e] < 0.f), fine = !odd_bits(v[e]);
            if (there && !fine) odd |= 1u << e;
            v[e] = there && fine ? v[e] : 0.f;
        }
        return v;
    };
    const float nan = __builtin_nanf("");
    Op<T> hs[KS];
    auto split_state = [&]() {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if (N < 32) hf[ks] = sel8(has, hf[ks]);
            split(hf[ks], hs[ks]);
        }
    };

    if constexpr (ONE) {
        const int nk = (K + 15) >> 4;
        const float* gc = reinterpret_cast<const float*>(smem + at.gc);
        const float* gb = reinterpret_cast<const float*>(smem + at.gb);
        for (int hh = 0; hh < nh; ++hh) {
            const int h = h0 + hh;
            const T* x = static_cast<const T*>(a.x) + row0 * a.xs + h * P + p0;
            T* y = static_cast<T*>(a.y) + (row0 * H + h) * P + p0;
            if (hh > 0) {
                load_state(h);
                __syncthreads();  // the tables are free
            }
            f32x4 xr[4];
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) xr[kt] = kt < nk ? load_x(x, a.xs, 16 * kt, K, lane, sel, upper) : zero4;
            for (int kt = w; kt < nk; kt += waves)
                tables(hh, kt, 16 * kt, 0, kt + 1, true, [&](int jt, f32x4& c, f32x4& b) {
                    const int tile = (kt * (kt + 1) / 2 + jt) * 256 + lane * 4;
                    c = ld4(gc + tile);
                    if (DELTA) b = ld4(gb + tile);
                });
            __syncthreads();
            u64 badx = 0;
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
                if (kt < nk) {
                    unsigned odd;
                    xr[kt] = clean_x(xr[kt], hh, 16 * kt, odd);
                    if (__ballot(odd != 0)) badx |= (u64)odd << (16 * kt + 4 * q);
                }
            if (__ballot(badx != 0)) {  // (a column's nodes are spread over its four lanes)
                badx |= __shfl_xor(badx, 16, 64);
                badx |= __shfl_xor(badx, 32, 64);
            }
            split_state();
            const float D = a.D ? a.D[h] : 0.f;
            F8 xf[2];
            Op<T> uf[2];
            f32x4 u[4] = {zero4, zero4, zero4, zero4};
            if (!DELTA) {
                xf[0] = pair8(x, xr[0], xr[1]);
                xf[1] = pair8(x, xr[2], xr[3]);
            } else {
                split(join(zero4, zero4), uf[0]);
                split(join(zero4, zero4), uf[1]);
            }
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
                if (kt < nk) {
                    const int k0 = 16 * kt;
                    const T* mt = reinterpret_cast<const T*>(smem + at.m + TreeLds::at(kt, true));
                    f32x4 o = zero4, v = zero4;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        o = mul(o, frag(Cm, a.cs, k0 + l16, ks), hs[ks]);
                        if (DELTA) v = mul(v, frag(Bm, a.bs, k0 + l16, ks), hs[ks]);
                    }
                    const f32x4 e4 = ld4(decay + hh * 64 + k0 + 4 * q);
                    o *= e4;
                    if constexpr (DELTA) {
                        const T* tt = reinterpret_cast<const T*>(smem + at.t + TreeLds::at(kt, true));
                        const f32x4 b4 = ld4(betas + hh * 64 + k0 + 4 * q);
                        f32x4 r;
#pragma unroll
                        for (int e = 0; e < 4; ++e) r[e] = e4[e] < 0.f ? 0.f : b4[e] * (xr[kt][e] - e4[e] * v[e]);
                        f32x4 t = zero4;
#pragma unroll
                        for (int f = 0; f < 2; ++f)
                            if (2 * f < kt) t = mul(t, get(tt, f, lane), uf[f]);
                        u[kt] = times_inv(reinterpret_cast<const T*>(smem + at.inv + kt * 1024), lane, r - t);
                        split(join(u[kt & ~1], u[kt | 1]), uf[kt >> 1]);
                    }
#pragma unroll
                    for (int f = 0; f < 2; ++f)
                        if (2 * f <= kt) {
                            if constexpr (DELTA) o = mul(o, get(mt, f, lane), uf[f]);
                            else o = mul(o, get(mt, f, lane), xf[f]);
                        }
                    settle(o);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (!DELTA) o[e] += D * xr[kt][e];
                        o[e] = e4[e] == -1.f ? 0.f : e4[e] == -2.f ? nan : o[e];
                    }
                    if (__ballot(badx != 0)) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!(e4[e] < 0.f) && (mask[k0 + 4 * q + e] & badx)) o[e] = nan;
                    }
                    store_y(y, ys, k0, K, lane, sel, upper, o);
                }
        }
    } else {
        const int h = h0;
        const T* x = static_cast<const T*>(a.x) + row0 * a.xs + h * P + p0;
        T* y = static_cast<T*>(a.y) + (row0 * H + h) * P + p0;
        u64* badx = reinterpret_cast<u64*>(smem + at.badx);
        const float D = a.D ? a.D[h] : 0.f;
        bool anybad = false;
        auto take_x = [&](int k0) {
            if (k0 >= K) return zero4;
            unsigned odd;
            const f32x4 v = clean_x(load_x(x, a.xs, k0, K, lane, sel, upper), 0, k0, odd);
            if (__ballot(odd != 0)) {
                anybad = true;
                if (odd) atomicOr(&badx[((k0 >> 6) * waves + w) * 16 + l16], (u64)odd << ((k0 & 63) + 4 * q));
                wave_sync();
            }
            return v;
        };
        split_state();
        for (int s = 0; s < panels; ++s) {
            const int q0 = s * kPanel, nk = (K - q0 + 15) / 16 < 4 ? (K - q0 + 15) / 16 : 4;
            f32x4 O[4], R[4], xt[4];
            // ---- what the held state gives: O = diag(E) C h^T, R = beta (x - diag(E) B h^T) ----
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                O[kt] = R[kt] = xt[kt] = zero4;
                if (kt < nk) {
                    const int k0 = q0 + 16 * kt;
                    f32x4 o = zero4, v = zero4;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        o = mul(o, frag(Cm, a.cs, k0 + l16, ks), hs[ks]);
                        if (DELTA) v = mul(v, frag(Bm, a.bs, k0 + l16, ks), hs[ks]);
                    }
                    const f32x4 e4 = ld4(decay + k0 + 4 * q);
                    settle(o);
                    O[kt] = e4 * o;
                    xt[kt] = take_x(k0);
                    if (DELTA) {
                        const f32x4 b4 = ld4(betas + k0 + 4 * q);
                        settle(v);
#pragma unroll
                        for (int e = 0; e < 4; ++e) R[kt][e] = e4[e] < 0.f ? 0.f : b4[e] * (xt[kt][e] - e4[e] * v[e]);
                    }
                }
            }
            for (int sp = 0; sp <= s; ++sp) {
                const bool own = sp == s;
                const int j0 = sp * kPanel;
                if (s > 0) __syncthreads();  // the tables are free
                for (int kt = w; kt < nk; kt += waves) {
                    F8 cf[KS], bf[KS];
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        cf[ks] = frag(Cm, a.cs, q0 + 16 * kt + l16, ks);
                        if (DELTA) bf[ks] = frag(Bm, a.bs, q0 + 16 * kt + l16, ks);
                    }
                    tables(0, kt, q0 + 16 * kt, j0, own ? kt + 1 : 4, own, [&](int jt, f32x4& c, f32x4& b) {
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) {
                            const F8 bj = frag(Bm, a.bs, j0 + 16 * jt + l16, ks);
                            c = mma(c, bj, cf[ks]);
                            if (DELTA) b = mma(b, bj, bf[ks]);
                        }
                        settle(c);
                        if (DELTA) settle(b);
                    });
                }
                __syncthreads();
                // ---- panel sp's part of R and O ----
                if constexpr (!DELTA) {
                    F8 xf[2];
#pragma unroll
                    for (int f = 0; f < 2; ++f)
                        xf[f] = own ? pair8(x, xt[2 * f], xt[2 * f + 1])
                                    : pair8(x, take_x(j0 + 32 * f), take_x(j0 + 32 * f + 16));
#pragma unroll
                    for (int kt = 0; kt < 4; ++kt)
                        if (kt < nk) {
                            const T* mt = reinterpret_cast<const T*>(smem + at.m + TreeLds::at(kt, false));
                            O[kt] = mul(O[kt], get(mt, 0, lane), xf[0]);
                            if (!own || kt >= 2) O[kt] = mul(O[kt], get(mt, 1, lane), xf[1]);
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
                                const T* tt = reinterpret_cast<const T*>(smem + at.t + TreeLds::at(kt, false));
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
#pragma unroll
                        for (int kt = 0; kt < 4; ++kt)
                            if (kt < nk) {
                                const T* tt = reinterpret_cast<const T*>(smem + at.t + TreeLds::at(kt, false));
                                f32x4 t = mul(mul(zero4, get(tt, 0, lane), uf[0]), get(tt, 1, lane), uf[1]);
                                settle(t);
                                R[kt] -= t;
                            }
                    }
#pragma unroll
                    for (int kt = 0; kt < 4; ++kt)
                        if (kt < nk) {
                            const T* mt = reinterpret_cast<const T*>(smem + at.m + TreeLds::at(kt, false));
                            O[kt] = mul(O[kt], get(mt, 0, lane), uf[0]);
                            if (!own || kt >= 2) O[kt] = mul(O[kt], get(mt, 1, lane), uf[1]);
                            settle(O[kt]);
                        }
                }
            }
            // ---- y ----
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
                    }
                    if (anybad) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            u64 hit = 0;  // a bad x on the node's path
                            for (int i = 0; i <= s; ++i) hit |= mask[(k0 + 4 * q + e) * panels + i] & badx[(i * waves + w) * 16 + l16];
                            if (hit && !(e4[e] < 0.f)) v[e] = nan;
                        }
                    }
                    store_y(y, ys, k0, K, lane, sel, upper, v);
                }
        }
    }
}

// Heads of a group that a work-group takes one after another (the paths and the products of B with C and
// itself are formed once for them), while that leaves every CU four work-groups.
inline int tree_heads(const Args& a, int slabs) {
    if (a.T > kPanel) return 1;
    const int hg = a.H / a.G;
    int hb = 8;
    while (hb > 1 && (hb > hg || a.b * a.G * ((hg + hb - 1) / hb) * slabs < 1024)) --hb;
    return hb;
}

template <typename T, int N>
int run_tree_n(const Args& a) {
    const int waves = a.P < 64 ? a.P / 16 : 4, slabs = a.P / (16 * waves);
    const int hb = tree_heads(a, slabs), hg = a.H / a.G;
    const bool one = a.T <= kPanel;
    const size_t lds = (size_t)TreeLds(one ? kPanel : (int)a.T, waves, hb, a.beta != nullptr).total;
    auto kernel = a.beta ? (one ? k_tree<T, N, true, true> : k_tree<T, N, true, false>)
                         : (one ? k_tree<T, N, false, true> : k_tree<T, N, false, false>);
    if (!delta::lds_limit(kernel, lds)) return 7;
    kernel<<<(unsigned)(a.b * a.G * ((hg + hb - 1) / hb) * slabs), 64 * waves, lds, a.stream>>>(a, hb);
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
