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
// A wave has 16 columns of headdim of one head; the state's rows are operand fragments straight from
// memory, and accumulators (rows 4 (l / 16) + e of a node tile, column l % 16) feed the next product as
// operands whose k index runs 16 (e / 4) + 4 (l / 16) + e % 4, so u never leaves its wave.  The waves of a
// work-group share the forming of M and T (B B^T and B C^T on the matrix cores, weighted by the decays), which
// reach them through LDS.  Up to 64 nodes (k_tree) the heads of a group follow each other in a work-group that
// keeps B's products; longer trees (k_tree_long) go 64 nodes at a time against panels of 64 up to their own.
//
// What bounds it.  A batch of trees reads each state once and each x, y once: 64 trees of 64 nodes, 80 heads of
// 64, dstate 128 move 255 MB in 67 us, 3.8 TB/s of reads and writes mixed (a large copy: 5.2), with the
// setup of a work-group (paths, decays, the first state: 13 to 22 thousand cycles, the last of which wait for memory)
// overlapped with its neighbours only.  Long trees are bound inside the CU: of 84 us for 16 lines of 200 nodes, 32 heads
// of 64, dstate 256, the delta rule, the table rows take 40% (the decays' exponentials and the splitting in two terms on
// the vector ALU), the reads of tables and rows from LDS 30%; memory would need 17 us.
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
__device__ __forceinline__ bf16x8 get_inv(const bf16* tab, int lane) { return ld8(tab + lane * 8); }
__device__ __forceinline__ f32x4 get_inv(const float* tab, int lane) { return ld4(tab + lane * 4); }
__device__ __forceinline__ f32x4 times_inv(bf16x8 a, f32x4 v) {
    bf16x4 o[2];
    delta::split4<2>(v, o);
    const bf16x4 zero = {};
    return mma(mma(f32x4{0.f, 0.f, 0.f, 0.f}, a, join(o[1], zero)), a, join(o[0], o[0]));
}
__device__ __forceinline__ f32x4 times_inv(f32x4 a, f32x4 v) { return delta::mma16(f32x4{0.f, 0.f, 0.f, 0.f}, a, v); }

constexpr int kTableBytes = 4096;  // of a node tile's M (or T) against a panel

// Up to 64 nodes: NK tiles of 16.  C's rows are kept in LDS as operand fragments for the products with the
// state, and B's where the delta rule needs them too; the scan has B's rows there only until B C^T is formed (in M's place).
template <typename T, int N, bool DELTA, int NK>
struct TreeCfg {
    static constexpr int KS = N < 32 ? 1 : N / 32;
    static constexpr int ROWS = NK * KS * 512 * (int)sizeof(T);  // bytes of C's or B's fragments
    // Waves a SIMD at least: three where the registers suffice without spills (32 trees of 40 nodes, wide heads, the
    // delta rule: 30.9 us, with two 35.3).
    static constexpr int WAVES = DELTA && NK < 4 && KS * (int)sizeof(T) <= 8 && sizeof(T) == 2 ? 3 : 1;
    static constexpr bool LCB = ROWS * (DELTA ? 2 : 1) <= 65536;
    static constexpr int TAB = NK == 1 ? 2048 : NK == 2 ? 4096 : NK == 3 ? 8192 : 12288;
    static constexpr int M = 0;                                                   // [tile] M as fragments
    static constexpr int TT = M + TAB;                                            // [tile] T
    static constexpr int INV = TT + (DELTA ? TAB : 0);                            // [tile] the diagonal tiles' inverses
    static constexpr int GC = DELTA ? INV + NK * 1024 : TAB > ROWS ? TAB : ROWS;  // [tile pair] the scan's B C^T
    static constexpr int CF = GC + (DELTA ? 0 : NK * (NK + 1) / 2 * 1024);        // C's rows
    static constexpr int BF = DELTA ? CF + (LCB ? ROWS : 0) : 0;                  // B's rows
    static constexpr int MASK = DELTA ? BF + (LCB ? ROWS : 0) : CF + ROWS;        // [node] the node and those above it
    static constexpr int BADB = MASK + 512;                                       // [tile] nodes whose row of B is not finite
    static constexpr int C = BADB + 64;  // [head][node] binary orders of decay from the held state
    static constexpr int HEAD = 64 * (8 + 4 + (DELTA ? 4 : 0));  // C, then E (-1 absent, -2 not computable), then beta
    static constexpr int total(int hb) { return C + hb * HEAD; }
    // tile kt's table: two KiB for each pair of tiles up to its own
    static __device__ int at(int kt) { return kt < 2 ? kt * 2048 : (kt - 1) * kTableBytes; }
};

// More nodes, in panels of 64.  kp: nodes rounded up to panels.  Where they fit (STG; not float32 at dstate 256), the rows
// of the panel in work go through LDS: x1 holds its C, then B of one earlier panel after another; x2 its own B (with
// one head and four waves a work-group: staged 226 us, every product's rows from memory 298).
template <typename T, int N, bool DELTA>
struct LongCfg {
    static constexpr int KS = N < 32 ? 1 : N / 32;
    static constexpr int ROWS = 4 * KS * 512 * (int)sizeof(T);
    static constexpr bool STG = 2 * ROWS <= 65536;
    static constexpr int KC = KS * (int)sizeof(T) <= 8 ? KS : 8 / (int)sizeof(T);  // fragments asked for at a time
    static constexpr int CH = KS / KC;                                             // such chunks of a tile's rows
    static constexpr int KH = KS > 1 ? KS / 2 : 1;               // a wave's share of an earlier panel's tile
};
struct LongLds {
    int tt, inv, x1, x2, mask, c, e, beta, badx, badb, more, total;  // M at 0: [head][tile], as T
    __host__ __device__ LongLds(int K, int heads, int cols, bool rule_delta, int rows) {
        const int kp = (K + kPanel - 1) / kPanel * kPanel, panels = kp / kPanel, tabs = heads * 4 * kTableBytes;
        tt = tabs;
        inv = tt + (rule_delta ? tabs : 0);  // [head][tile] the diagonal tiles' inverses
        x1 = inv + (rule_delta ? heads * 4096 : 0);
        x2 = x1 + rows;
        mask = x2 + rows;              // [panel][node]
        c = mask + kp * panels * 8;    // [head][node], as E and beta
        e = c + heads * kp * 8;
        beta = e + heads * kp * 4;
        badx = beta + (rule_delta ? heads * kp * 4 : 0);  // [panel][wave with columns][column] nodes whose x is not finite
        badb = badx + panels * heads * cols * 16 * 8;     // [tile] nodes whose row of B is not finite
        more = badb + 64;  // [round] whether paths go on
        total = more + 64;
    }
};

__device__ __forceinline__ bool odd_bits(float v) { return (__builtin_bit_cast(unsigned, v) & 0x7f800000u) == 0x7f800000u; }
// Whether an element of v is not finite, its exponent's bits all ones: one more carries into the sign's place.
__device__ __forceinline__ unsigned odd_carry(bf16x8 v) {
    const u32x4v w = (__builtin_bit_cast(u32x4v, v) & 0x7f807f80u) + 0x00800080u;
    return (w[0] | w[1] | w[2] | w[3]) & 0x80008000u;
}
__device__ __forceinline__ unsigned odd_carry(f32x8 v) {
    typedef unsigned u32x8v __attribute__((ext_vector_type(8)));
    const u32x8v w = (__builtin_bit_cast(u32x8v, v) & 0x7f800000u) + 0x00800000u;
    return (w[0] | w[1] | w[2] | w[3] | w[4] | w[5] | w[6] | w[7]) & 0x80000000u;
}
// orders LDS traffic of one wave's lanes (LDS serves a wave in order; this keeps the compiler to it)
__device__ __forceinline__ void wave_sync() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// All of v has arrived here: its reads go out together ahead of this, and not one by one between the products
// (which cost an LDS latency each).
template <typename F8, int KS>
__device__ __forceinline__ void together(F8 (&v)[KS]) {
    if constexpr (KS == 1) asm volatile("" : "+v"(v[0]));
    else if constexpr (KS == 2) asm volatile("" : "+v"(v[0]), "+v"(v[1]));
    else if constexpr (KS == 4) asm volatile("" : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]));
    else asm volatile("" : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]), "+v"(v[7]));
}

__device__ __forceinline__ void together(Op<bf16>& a) { asm volatile("" : "+v"(a.t[0]), "+v"(a.t[1])); }
__device__ __forceinline__ void together(Op<float>& a) { asm volatile("" : "+v"(a.t[0])); }

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

// A node tile's x and y as accumulators hold them (lane: nodes 4 q + e, column l % 16).  bfloat16 moves 8
// bytes a lane through a transpose in the ALU.  Rows past the last node read as the last, and drop stores.
template <typename T> struct Raw;
template <> struct Raw<bf16> { typedef delta::u32x2v type; };
template <> struct Raw<float> { typedef f32x4 type; };
__device__ __forceinline__ delta::u32x2v load_x(const bf16* x, int64_t xs, int k0, int K, int lane) {
    const int k = k0 + 4 * (lane >> 4) + (lane & 3);
    return *reinterpret_cast<const delta::u32x2v*>(x + (int64_t)(k < K ? k : K - 1) * xs + 4 * ((lane & 15) >> 2));
}
__device__ __forceinline__ f32x4 load_x(const float* x, int64_t xs, int k0, int K, int lane) {
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int k = k0 + 4 * (lane >> 4) + e;
        v[e] = x[(int64_t)(k < K ? k : K - 1) * xs + (lane & 15)];
    }
    return v;
}
__device__ __forceinline__ f32x4 open_x(delta::u32x2v v, unsigned sel, bool upper) { return delta::floats(delta::quad_t(v, sel, upper)); }
__device__ __forceinline__ f32x4 open_x(f32x4 v, unsigned, bool) { return v; }
// y: the row's first element of this wave's columns; rs: elements between nodes (16 of them within 2 GiB)
template <typename T>
__device__ __forceinline__ brsrc y_tile(T* y, int64_t rs, int k0, int K) {
    const int n = K - k0 < 16 ? K - k0 : 16;
    return make_rsrc(y + (int64_t)k0 * rs, n > 0 ? (uint32_t)(((n - 1) * rs + 16) * (int64_t)sizeof(T)) : 0u);
}
__device__ __forceinline__ void store_y(bf16* y, int64_t rs, int k0, int K, int lane, unsigned sel, bool upper, f32x4 v) {
    const delta::u32x2v w = delta::quad_t(delta::u32x2v{delta::cvt2(v[0], v[1]), delta::cvt2(v[2], v[3])}, sel, upper);
    const int off = ((4 * (lane >> 4) + (lane & 3)) * (int)rs + 4 * ((lane & 15) >> 2)) * 2;
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, w), y_tile(y, rs, k0, K), off, 0, 0);
}
__device__ __forceinline__ void store_y(float* y, int64_t rs, int k0, int K, int lane, unsigned, bool, f32x4 v) {
    const brsrc r = y_tile(y, rs, k0, K);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, (float)v[e]), r, ((4 * (lane >> 4) + e) * (int)rs + (lane & 15)) * 4, 0, 0);
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

typedef unsigned long long u64;

// Which (row, group, heads, columns) a work-group takes; cols: its waves that have columns (the others get addresses of
// theirs, so that loads need no branch: behind one the compiler waits for everything that may be on its way).  Blocks
// k, k + 8, ... run on one XCD: each takes a contiguous range, so that a row's B, C and dt stay in its L2.
struct Place {
    int64_t bi;
    int g, h0, nh, p0;
    __device__ Place(const Args& a, int hb, int cols, int w) {
        const unsigned hg = a.H / a.G, slabs = a.P / (16 * cols), chunks = (hg + hb - 1) / hb, nb = gridDim.x;
        unsigned id = nb % 8 == 0 ? blockIdx.x % 8 * (nb / 8) + blockIdx.x / 8 : blockIdx.x;
        p0 = ((int)(id % slabs) * cols + w % cols) * 16;
        id /= slabs;
        const unsigned chunk = id % chunks;
        id /= chunks;
        g = (int)(id % a.G);
        bi = id / a.G;
        h0 = (int)(g * hg + chunk * hb);
        nh = (int)(hg - chunk * hb < (unsigned)hb ? hg - chunk * hb : hb);
    }
};

// A node tile's table row from its products and decays; bits: which of the lane's nodes 4 q + e are on the path of
// node k; ck, cj: their orders.  A row that two waves share: one table's; or a wave's alone: M's (of c) and T's (of b).
__device__ __forceinline__ f32x4 weigh(unsigned bits, double ck, const double* cj, float scale, f32x4 c) {
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float f = exp2f_fast((float)(ck - cj[e]));
        v[e] = bits >> e & 1 ? scale * f * c[e] : 0.f;
    }
    return v;
}
template <bool DELTA>
__device__ __forceinline__ void weigh(unsigned bits, double ck, const double* cj, float bk, int self, f32x4 c, f32x4 b,
                                      f32x4& m, f32x4& t) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float f = exp2f_fast((float)(ck - cj[e]));
        const bool on = bits >> e & 1;
        m[e] = on ? f * c[e] : 0.f;
        if (DELTA) t[e] = on && e != self ? bk * f * b[e] : 0.f;
    }
}

// x of a tile with zeros for absent nodes and for values that are not finite; the latter's nodes
// (bits e) come back in `odd`
__device__ __forceinline__ f32x4 clean_x(f32x4 v, const float* decay4, unsigned& odd) {
    const f32x4 e4 = ld4(decay4);
    odd = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bool there = !(e4[e] < 0.f), fine = !odd_bits(v[e]);
        if (there && !fine) odd |= 1u << e;
        v[e] = there && fine ? v[e] : 0.f;
    }
    return v;
}

// ---------------------------------------------------------------------------
// k_tree: trees of up to 16 NK nodes.  A work-group takes hb heads of a group one after another: paths, the
// products of B with C and itself, and the rows of C and B are formed or fetched once for them.  Wave w forms the tables
// of node tile w (w < NK) and has 16 columns (w < cols).  Per head: tables, a barrier, then each wave's columns tile by
// tile from LDS alone, while the next head's state and x are on their way: no load is waited for behind a store of y.
// Times: one tree of 8 nodes over 48 heads of 64, dstate 128 6.0 us (a chain of latencies: parents and slot, the
// state, tables, products); 64 trees of 64 nodes, 80 heads 67 us; 32 trees of 40 nodes, 32 heads of 128, 16 groups, the
// delta rule 31 us (k_tree_long, which has the 64 nodes in one panel, would need 113 and 52).
// ---------------------------------------------------------------------------
template <typename T, int N, bool DELTA, int NK>
__global__ __launch_bounds__(256, (TreeCfg<T, N, DELTA, NK>::WAVES)) void k_tree(Args a, int hb) {
    typedef typename V8<T>::type F8;
    typedef TreeCfg<T, N, DELTA, NK> CF;
    constexpr int KS = CF::KS;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int waves = blockDim.x >> 6, K = (int)a.T, P = a.P, H = a.H, cols = P < 64 ? P / 16 : 4;
    const int w = wave_id();
    int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    // addresses are formed again where they are used: kept over the loop they would take the registers of operands
    auto again = [&] {
        asm volatile("" : "+v"(lane));
        l16 = lane & 15;
        q = lane >> 4;
    };
    const Place at(a, hb, cols, w);
    const int64_t row0 = at.bi * K, ys = (int64_t)H * P;
    const unsigned sel = delta::quad_sel(lane);
    const bool upper = (lane & 2) != 0, mine = w < cols, tiled = w < NK;
    T* mtab = reinterpret_cast<T*>(smem + CF::M);
    T* ttab = reinterpret_cast<T*>(smem + CF::TT);
    float* gc = reinterpret_cast<float*>(smem + CF::GC);
    T* crow = reinterpret_cast<T*>(smem + CF::CF);
    T* brow = reinterpret_cast<T*>(smem + CF::BF);
    u64* mask = reinterpret_cast<u64*>(smem + CF::MASK);
    u64* badb = reinterpret_cast<u64*>(smem + CF::BADB);
    float* skips = reinterpret_cast<float*>(smem + CF::BADB);  // [head] the scan's D (which has no use for badb)
    double* cs = reinterpret_cast<double*>(smem + CF::C);
    float* decay = reinterpret_cast<float*>(smem + CF::C + hb * 512);
    float* betas = reinterpret_cast<float*>(smem + CF::C + hb * 768);
    const T* Bm = static_cast<const T*>(a.B) + row0 * a.bs + at.g * N;
    const T* Cm = static_cast<const T*>(a.C) + row0 * a.cs + at.g * N;
    const T* beta = static_cast<const T*>(a.beta);
    const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
    const int slot = a.slots[at.bi];
    const bool has = N >= 32 || q < 2;  // (dstate 16 fills half a fragment)
    const int n0 = 8 * (N >= 32 ? q : q & 1);
    // the state's rows as operands: lane (q, l16) holds row p0 + l16, elements 32 ks + 8 q .. + 7; and x
    f32x8 hf[KS];
    typename Raw<T>::type xq[NK];
    auto fetch = [&](int h) {
        const float* hp = a.pool + slot * a.ss + (int64_t)(h * P + at.p0 + l16) * N + n0;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) hf[ks] = ld8(hp + 32 * ks);
        const T* x = static_cast<const T*>(a.x) + row0 * a.xs + h * P + at.p0;
#pragma unroll
        for (int kt = 0; kt < NK; ++kt) xq[kt] = load_x(x, a.xs, 16 * kt, K, lane);
    };
    // row `node` (rows past the last are never used) of B or C
    auto frag = [&](const T* m, int64_t stride, int node, int ks) {
        const F8 v = ld8(m + (int64_t)(node < K ? node : K - 1) * stride + 32 * ks + n0);
        return N >= 32 ? v : sel8(has, v);
    };
    auto kept = [&](const T* rows, int tile, int ks) { return ld8(rows + ((tile * KS + ks) * 64 + lane) * 8); };

    // ---- what the heads share, and every head's decays ----
    const int par = lane < K ? a.parents[row0 + lane] : -2;
    float dtv[2], btv[2];  // of the wave's first two heads
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int hh = w + i * waves < at.nh ? w + i * waves : 0;
        const int64_t k = (row0 + (lane < K ? lane : K - 1)) * H + at.h0 + hh;
        dtv[i] = a.dt[k];
        btv[i] = DELTA ? to_f(beta[k]) : 0.f;
    }
    const float skip = !DELTA && a.D ? a.D[at.h0 + (lane < at.nh ? lane : 0)] : 0.f;
    F8 cf[KS], bf[KS];  // the rows of this wave's node tile
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        cf[ks] = frag(Cm, a.cs, 16 * w + l16, ks);
        bf[ks] = frag(Bm, a.bs, 16 * w + l16, ks);
    }
    // (all of the above is on its way before the slot is looked at)
    if (slot < 0 || slot >= a.S) {
        if (mine)
            for (int hh = 0; hh < at.nh; ++hh)
                for (int k0 = 0; k0 < K; k0 += 16)
                    store_y(static_cast<T*>(a.y) + (row0 * H + at.h0 + hh) * P + at.p0, ys, k0, K, lane, sel, upper, zero4);
        return;
    }
    f32x4 gcr[NK], gbr[NK];  // the delta rule's B C^T and B B^T of this wave's node tile
#pragma unroll
    for (int jt = 0; jt < NK; ++jt) gcr[jt] = gbr[jt] = zero4;
    fetch(at.h0);  // (behind what the products wait for)
    if (tiled) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if (CF::LCB) st8(crow + ((w * KS + ks) * 64 + lane) * 8, cf[ks]);
            if (CF::LCB || !DELTA) st8(brow + ((w * KS + ks) * 64 + lane) * 8, bf[ks]);
        }
    }
    __syncthreads();
    if (tiled) {
#pragma unroll
        for (int jt = 0; jt < NK; ++jt)
            if (jt <= w) {
                f32x4 c = zero4, b = zero4;
                F8 bj[KS];
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) bj[ks] = CF::LCB || !DELTA ? kept(brow, jt, ks) : frag(Bm, a.bs, 16 * jt + l16, ks);
                together(bj);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    c = mma(c, bj[ks], cf[ks]);
                    if (DELTA) b = mma(b, bj[ks], bf[ks]);
                }
                settle(c);
                if (DELTA) {
                    settle(b);
                    gcr[jt] = c;
                    gbr[jt] = b;
                    if (jt == w) {
                        // |B_k|^2 on the diagonal is finite where the row is, unless the square leaves float32: then its
                        // elements tell (looked at always they spill at three waves a SIMD: tree of 40 nodes above 34.0 us, so 30.7)
                        const float d = l16 & 2 ? (l16 & 1 ? b[3] : b[2]) : (l16 & 1 ? b[1] : b[0]);
                        u64 who = __ballot(q == l16 >> 2 && odd_bits(d));
                        who |= who >> 32;
                        who = (who | who >> 16) & 0xffff;
                        if (who) {
                            unsigned odd = 0;
#pragma unroll 1
                            for (int ks = 0; ks < KS; ++ks) odd |= odd_carry(CF::LCB ? kept(brow, w, ks) : frag(Bm, a.bs, 16 * w + l16, ks));
                            who = __ballot(odd != 0);
                            who |= who >> 32;
                            who = (who | who >> 16) & 0xffff;
                        }
                        if (lane == 0) badb[w] = who << (16 * w);
                    }
                } else {
                    st4(gc + (w * (w + 1) / 2 + jt) * 256 + lane * 4, c);
                }
            }
    }
    // the paths, by doubling: pr[r] is the node 2^r above
    bool there = lane < K && par >= -1 && par < lane;
    u64 mk = 1ull << lane;
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
    if (w == 0) {
        mask[lane] = mk;
        if (!DELTA && lane < 16) skips[lane] = skip;
    }
    if (DELTA) __syncthreads();
    for (int i = 0, hh = w; hh < at.nh; ++i, hh += waves) {
        float dt = dtv[0], bt = btv[0];
        if (i == 1) dt = dtv[1], bt = btv[1];
        if (i > 1) {
            const int64_t k = (row0 + (lane < K ? lane : K - 1)) * H + at.h0 + hh;
            dt = a.dt[k];
            if (DELTA) bt = to_f(beta[k]);
        }
        double c = orders(dt, (double)a.A[at.h0 + hh] * 1.4426950408889634);
        bool bad = false;
        if (DELTA) {
            u64 odd = __ballot(c != c || odd_bits(bt));
#pragma unroll
            for (int kt = 0; kt < NK; ++kt) odd |= badb[kt];
            bad = (mk & odd) != 0;
            betas[hh * 64 + lane] = bt;
        }
#pragma unroll
        for (int r = 0; r < 6; ++r)
            if (r < rounds) {
                const double up = __shfl(c, pr[r] < 0 ? lane : pr[r], 64);
                if (pr[r] >= 0) c += up;
            }
        cs[hh * 64 + lane] = c;
        decay[hh * 64 + lane] = !there ? -1.f : bad ? -2.f : exp2f_fast((float)c);
    }
    __syncthreads();

    const float nan = __builtin_nanf("");
    for (int hh = 0; hh < at.nh; ++hh) {
        again();
        const int h = at.h0 + hh;
        // ---- M and T of this wave's node tile ----
        if (tiled) {
            T* mt = mtab + CF::at(w) / (int)sizeof(T);
            T* tt = ttab + CF::at(w) / (int)sizeof(T);
            const int k = 16 * w + l16;
            const u64 on = decay[hh * 64 + k] < 0.f ? 0 : mask[k];
            const double ck = cs[hh * 64 + k];
            const float bk = DELTA ? betas[hh * 64 + k] : 0.f;
            f32x4 diag = zero4;
#pragma unroll
            for (int jt = 0; jt < ((NK + 1) & ~1); ++jt)
                if (jt < ((w + 2) & ~1)) {
                    f32x4 m = zero4, t = zero4;
                    if (jt < NK && jt <= w) {
                        f32x4 c;
                        if (DELTA) c = gcr[jt < NK ? jt : 0];
                        else c = ld4(gc + (w * (w + 1) / 2 + jt) * 256 + lane * 4);
                        weigh<DELTA>((unsigned)(on >> (16 * jt + 4 * q)) & 15u, ck, cs + hh * 64 + 16 * jt + 4 * q, bk,
                                     k - 16 * jt - 4 * q, c, gbr[jt < NK ? jt : 0], m, t);
                    }
                    put(mt, jt >> 1, jt & 1, lane, m);
                    if (DELTA) {
                        if (jt == w) {
                            diag = t;
                            t = zero4;
                        }
                        put(tt, jt >> 1, jt & 1, lane, t);
                    }
                }
            if (DELTA) {
                T* inv = reinterpret_cast<T*>(smem + CF::INV + w * 1024);
                put_inv(inv, lane, inverse16(diag, reinterpret_cast<float*>(inv), lane));
            }
        }
        __syncthreads();
        if (!mine) {
            if (hh + 1 < at.nh) __syncthreads();
            continue;
        }
        again();
        // ---- this head's operands; then the next head's are asked for ----
        f32x4 xr[NK];
        u64 badx = 0;
#pragma unroll
        for (int kt = 0; kt < NK; ++kt) {
            unsigned odd;
            xr[kt] = clean_x(open_x(xq[kt], sel, upper), decay + hh * 64 + 16 * kt + 4 * q, odd);
            badx |= (u64)odd << (16 * kt + 4 * q);
        }
        if (__ballot(badx != 0)) {  // (a column's nodes are spread over its four lanes)
            badx |= __shfl_xor(badx, 16, 64);
            badx |= __shfl_xor(badx, 32, 64);
        }
        Op<T> hs[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) split(N >= 32 ? hf[ks] : sel8(has, hf[ks]), hs[ks]);
        if (hh + 1 < at.nh) fetch(h + 1);
        T* y = static_cast<T*>(a.y) + (row0 * H + h) * P + at.p0;
        const float D = DELTA ? 0.f : skips[hh];
        F8 xf[(NK + 1) / 2];
        Op<T> uf[(NK + 1) / 2];
        f32x4 u[NK + 1];
#pragma unroll
        for (int kt = 0; kt <= NK; ++kt) u[kt] = zero4;
#pragma unroll
        for (int f = 0; f < (NK + 1) / 2; ++f) {
            if (!DELTA) xf[f] = pair8(y, xr[2 * f], 2 * f + 1 < NK ? xr[(2 * f + 1) % NK] : zero4);
            if (DELTA) split(join(zero4, zero4), uf[f]);
        }
#pragma unroll
        for (int kt = 0; kt < NK; ++kt) {
            const int k0 = 16 * kt;
            f32x4 o = zero4, v = zero4;
            F8 fr[KS];
            Op<T> mo[2], to[2];
            auto ask_tables = [&] {
#pragma unroll
                for (int f = 0; 2 * f <= kt; ++f) {
                    mo[f] = get(mtab + CF::at(kt) / (int)sizeof(T), f, lane);
                    if (DELTA && 2 * f < kt) to[f] = get(ttab + CF::at(kt) / (int)sizeof(T), f, lane);
                }
            };
            auto have_tables = [&] {
#pragma unroll
                for (int f = 0; 2 * f <= kt; ++f) {
                    together(mo[f]);
                    if (DELTA && 2 * f < kt) together(to[f]);
                }
            };
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) fr[ks] = CF::LCB ? kept(crow, kt, ks) : frag(Cm, a.cs, k0 + l16, ks);
            const f32x4 e4 = ld4(decay + hh * 64 + k0 + 4 * q);
            if (!DELTA) ask_tables();
            together(fr);
            if (!DELTA) have_tables();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) o = mul(o, fr[ks], hs[ks]);
            if constexpr (DELTA) {
                // B's rows take the registers of C's, and the tables theirs: a third wave a SIMD hides the wait
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) fr[ks] = CF::LCB ? kept(brow, kt, ks) : frag(Bm, a.bs, k0 + l16, ks);
                together(fr);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) v = mul(v, fr[ks], hs[ks]);
                ask_tables();
                have_tables();
            }
            o *= e4;
            if constexpr (DELTA) {
                const f32x4 b4 = ld4(betas + hh * 64 + k0 + 4 * q);
                const auto inv = get_inv(reinterpret_cast<const T*>(smem + CF::INV + kt * 1024), lane);
                f32x4 r;
#pragma unroll
                for (int e = 0; e < 4; ++e) r[e] = e4[e] < 0.f ? 0.f : b4[e] * (xr[kt][e] - e4[e] * v[e]);
                f32x4 t = zero4;
#pragma unroll
                for (int f = 0; 2 * f < kt; ++f) t = mul(t, to[f], uf[f]);
                u[kt] = times_inv(inv, r - t);
                split(join(u[kt & ~1], u[kt | 1]), uf[kt >> 1]);
            }
#pragma unroll
            for (int f = 0; 2 * f <= kt; ++f) {
                if constexpr (DELTA) o = mul(o, mo[f], uf[f]);
                else o = mul(o, mo[f], xf[f]);
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
        if (hh + 1 < at.nh) __syncthreads();  // the tables are free
    }
}

// ---------------------------------------------------------------------------
// k_tree_long: trees of 65 to 256 nodes, 64 nodes at a time against every panel of 64 up to their own.  Eight waves
// take one head, or two of a group (16 columns a wave).  For the tables, wave w has node tile w % 4 and one operand's
// rows: C's (waves 0 to 3, M) or B's (4 to 7, T); a product serves both heads, and the diagonal tiles' inverses go to the
// waves with the shorter rows of the own panel.  The scan has no T: its waves 4 to 7 take half of M's tiles.  u of
// earlier panels stays in registers, two terms as the next product takes them; no tile goes back to memory.
// 16 lines of 200 nodes, 32 heads of 64, 8 groups, dstate 256, the delta rule: 84 us (one head a work-group 129).
// ---------------------------------------------------------------------------
template <typename T, int N, bool DELTA>
__global__ __launch_bounds__(512) void k_tree_long(Args a, int heads) {
    typedef typename V8<T>::type F8;
    typedef LongCfg<T, N, DELTA> CF;
    constexpr int KS = CF::KS, KH = CF::KH, KC = CF::KC, CH = CF::CH;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int K = (int)a.T, P = a.P, H = a.H, cols = P / 16;
    const int tid = threadIdx.x, w = wave_id();
    int lane = tid & 63, l16 = lane & 15, q = lane >> 4;
    // addresses are formed again where they are used: kept over the loops they would take the registers of operands
    auto again = [&] {
        asm volatile("" : "+v"(lane));
        l16 = lane & 15;
        q = lane >> 4;
    };
    const int tw = w & 3, kind = w >> 2;  // of the tables
    const int hw = heads == 2 ? w >> 2 : 0, cw = heads == 2 ? w & 3 : w;  // of the columns
    const Place place(a, heads, cols, cw);
    const bool mine = hw < place.nh && cw < cols;
    const int64_t row0 = place.bi * K, ys = (int64_t)H * P;
    const int g = place.g, h = place.h0 + (mine ? hw : 0), p0 = place.p0;
    const unsigned sel = delta::quad_sel(lane);
    const bool upper = (lane & 2) != 0;
    const int kp = (K + kPanel - 1) / kPanel * kPanel, panels = kp / kPanel;
    const LongLds at(K, heads, cols, DELTA, CF::STG ? CF::ROWS : 0);
    T* mtabs = reinterpret_cast<T*>(smem);
    T* ttabs = reinterpret_cast<T*>(smem + at.tt);
    T* x1 = reinterpret_cast<T*>(smem + at.x1);
    T* x2 = reinterpret_cast<T*>(smem + at.x2);
    constexpr int TAB = kTableBytes / (int)sizeof(T);
    u64* mask = reinterpret_cast<u64*>(smem + at.mask);
    double* css = reinterpret_cast<double*>(smem + at.c);
    float* decays = reinterpret_cast<float*>(smem + at.e);
    float* betas = reinterpret_cast<float*>(smem + at.beta);
    int* ptr = reinterpret_cast<int*>(smem);  // [node], in M's place while the paths are formed
    u64* badx = reinterpret_cast<u64*>(smem + at.badx) + (mine ? (hw * cols + cw) * 16 + l16 : 0);
    const int badp = heads * cols * 16;       // from one panel's to the next
    unsigned* badb = reinterpret_cast<unsigned*>(smem + at.badb);
    unsigned* more = reinterpret_cast<unsigned*>(smem + at.more);
    // this wave's head's
    const T* mt = mtabs + (mine ? hw : 0) * 4 * TAB;
    const T* tt = ttabs + (mine ? hw : 0) * 4 * TAB;
    float* decay = decays + (mine ? hw : 0) * kp;
    const T* x = static_cast<const T*>(a.x) + row0 * a.xs + h * P + p0;
    const T* Bm = static_cast<const T*>(a.B) + row0 * a.bs + g * N;
    const T* Cm = static_cast<const T*>(a.C) + row0 * a.cs + g * N;
    const T* beta = static_cast<const T*>(a.beta);
    T* y = static_cast<T*>(a.y) + (row0 * H + h) * P + p0;
    const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
    const bool has = N >= 32 || q < 2;
    const int n0 = 8 * (N >= 32 ? q : q & 1);
    auto frag = [&](const T* m, int64_t stride, int node, int ks) {
        const F8 v = ld8(m + (int64_t)(node < K ? node : K - 1) * stride + 32 * ks + n0);
        return N >= 32 ? v : sel8(has, v);
    };
    auto kept = [&](const T* rows, int tile, int ks) { return ld8(rows + ((tile * KS + ks) * 64 + lane) * 8); };
    // the rows that this wave stages: node tile tw of a panel's C or B; and its share of an earlier panel's B
    const T* rows = kind ? Bm : Cm;
    const int64_t rows_st = kind ? a.bs : a.cs;
    F8 rs[KS];
    auto ask_own = [&](int j0) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) rs[ks] = frag(rows, rows_st, j0 + 16 * tw + l16, ks);
    };
    const int first = KS > 1 ? kind * KH : 0;
    auto ask_b = [&](int j0, F8 (&bn)[KH]) {
#pragma unroll
        for (int i = 0; i < KH; ++i) bn[i] = frag(Bm, a.bs, j0 + 16 * tw + l16, first + i);
    };
    auto keep_b = [&](const F8 (&bn)[KH]) {
        if (KS > 1 || kind == 0)
#pragma unroll
            for (int i = 0; i < KH; ++i) st8(x1 + ((tw * KS + first + i) * 64 + lane) * 8, bn[i]);
    };
    // a thread a node and head
    const int nt = tid & 255, ht = w >> 2;
    const bool in = nt < K;
    const int64_t node = row0 + (in ? nt : K - 1);
    const int hn = place.h0 + (ht < place.nh ? ht : 0);
    const float dt = a.dt[node * H + hn], bt = DELTA ? to_f(beta[node * H + hn]) : 0.f;
    const int par = a.parents[node];
    typename Raw<T>::type xq[4], xn[4];
    if (CF::STG) ask_own(0);
    const int slot = a.slots[place.bi];
    if (slot < 0 || slot >= a.S) {
        if (mine)
            for (int k0 = 0; k0 < K; k0 += 16) store_y(y, ys, k0, K, lane, sel, upper, zero4);
        return;
    }
    f32x8 hf[KS];  // (behind what the panels wait for)
    {
        const float* hp = a.pool + slot * a.ss + (int64_t)(h * P + p0 + l16) * N + n0;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) hf[ks] = ld8(hp + 32 * ks);
    }
    for (int i = tid; i < badp * panels; i += 512) reinterpret_cast<u64*>(smem + at.badx)[i] = 0;
    if (tid < 16) badb[tid] = more[tid] = 0;
    const bool sets = ht < place.nh && nt < kp;
    const int kn = ht * kp + nt;
    if (sets) {
        const double c = orders(in ? dt : 0.f, (double)a.A[hn] * 1.4426950408889634);
        const bool ok = in && par >= -1 && par < nt;
        if (DELTA) betas[kn] = in ? bt : 0.f;
        css[kn] = c;
        decays[kn] = !ok ? -1.f : DELTA && (c != c || odd_bits(bt)) ? -2.f : 0.f;
        if (ht == 0) {
            ptr[nt] = ok ? par : -1;
            for (int i = 0; i < panels; ++i) mask[i * kp + nt] = i == nt >> 6 ? 1ull << (nt & 63) : 0;
        }
    }
    __syncthreads();
    // the paths, by doubling; a node is absent below an absent one, and not computable below such a one
    for (int r = 0, reach = 1; reach < K; reach *= 2, ++r) {
        const int k = sets ? nt : 0, of = sets ? ht * kp : 0, p = ptr[k], from = p < 0 ? k : p;
        const double c = p < 0 ? css[of + k] : css[of + k] + css[of + from];
        const int up = p < 0 ? -1 : ptr[from];
        const float self = decays[of + k], theirs = decays[of + from];
        u64 m[4];
        if (ht == 0)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < panels) m[j] = mask[j * kp + k] | mask[j * kp + from];
        if (__ballot(up >= 0) && lane == 0) more[r] = 1;
        __syncthreads();
        if (sets) {
            css[kn] = c;
            decays[kn] = self == -1.f || theirs == -1.f ? -1.f : self < theirs ? self : theirs;
            if (ht == 0) {
                ptr[k] = up;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < panels) mask[j * kp + k] = m[j];
            }
        }
        __syncthreads();
        if (!more[r]) break;
    }
    if (sets && !(decays[kn] < 0.f)) decays[kn] = exp2f_fast((float)css[kn]);
    __syncthreads();

    const float nan = __builtin_nanf("");
    const float D = a.D ? a.D[h] : 0.f;
    bool anybad = false;
    auto ask_x = [&](int k0, typename Raw<T>::type (&v)[4]) {
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) v[kt] = load_x(x, a.xs, k0 + 16 * kt, K, lane);
    };
    auto take_x = [&](typename Raw<T>::type raw, int k0) {
        unsigned odd;
        const f32x4 v = clean_x(open_x(raw, sel, upper), decay + k0 + 4 * q, odd);
        if (__ballot(odd != 0)) {
            anybad = true;
            if (odd && mine) atomicOr(badx + (k0 >> 6) * badp, (u64)odd << ((k0 & 63) + 4 * q));
            wave_sync();
        }
        return v;
    };
    Op<T> hs[KS], u0[2], u1[2], u2[2];  // the state; u of the panels before the last
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) split(N >= 32 ? hf[ks] : sel8(has, hf[ks]), hs[ks]);
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        split(join(zero4, zero4), u0[f]);
        u2[f] = u1[f] = u0[f];
    }
    ask_x(0, xq);
#pragma unroll 1
    for (int s = 0; s < panels; ++s) {
        again();
        const int q0 = s * kPanel, nk = (K - q0 + 15) / 16 < 4 ? (K - q0 + 15) / 16 : 4;
        if (s > 0) __syncthreads();  // x1 and x2 are free
        if (CF::STG) {
            T* to = kind ? x2 : x1;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) st8(to + ((tw * KS + ks) * 64 + lane) * 8, rs[ks]);
        }
        if (DELTA && kind) {
            // a node below one whose row of B is not finite cannot be computed
            if (!CF::STG) ask_own(q0);
            unsigned odd = 0;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) odd |= odd_carry(rs[ks]);
            u64 who = __ballot(odd != 0);
            who |= who >> 32;
            if (lane == 0) badb[4 * s + tw] = (unsigned)(who | who >> 16) & 0xffffu;
        }
        __syncthreads();
        if (DELTA) {
            u64 odd[4];
            bool any = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // (zero for panels to come)
                odd[i] = badb[4 * i] | badb[4 * i + 1] << 16 | (u64)(badb[4 * i + 2] | badb[4 * i + 3] << 16) << 32;
                any |= odd[i] != 0;
            }
            if (any) {
                if (ht < place.nh && nt < kPanel) {
                    u64 hit = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i <= s) hit |= mask[i * kp + q0 + nt] & odd[i];
                    float& e = decays[ht * kp + q0 + nt];
                    if (hit && e != -1.f) e = -2.f;
                }
                __syncthreads();
            }
        }
        if (!DELTA && s > 0) ask_x(0, xn);
        f32x4 O[4], Rt[4], xt[4];
        // ---- what the held state gives: O = diag(E) C h^T, Rt = beta (x - diag(E) B h^T) ----
        constexpr int MATS = DELTA ? 2 : 1, STEPS = MATS * CH;  // chunks of a tile: C's, then B's
        F8 fr[2][KC];  // the chunk in work and the next
        auto ask = [&](int i) {
            const int kt = i / STEPS, mat = i / CH % MATS, c = i % CH;
#pragma unroll
            for (int ks = 0; ks < KC; ++ks)
                fr[i & 1][ks] = CF::STG ? kept(mat ? x2 : x1, kt, c * KC + ks)
                                        : frag(mat ? Bm : Cm, mat ? a.bs : a.cs, q0 + 16 * kt + l16, c * KC + ks);
        };
        ask(0);
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            const int k0 = q0 + 16 * kt;
            O[kt] = Rt[kt] = zero4;
            xt[kt] = take_x(xq[kt], k0);  // (zero past the last node)
            if (kt < nk && mine) {
                f32x4 ov[MATS][kTwo<T>];
#pragma unroll
                for (int j = 0; j < STEPS; ++j) {
                    const int i = kt * STEPS + j, mat = j / CH, c = j % CH;
                    together(fr[i & 1]);
                    if (i + 1 < 4 * STEPS) ask(i + 1);
#pragma unroll
                    for (int ks = 0; ks < KC; ++ks)
#pragma unroll
                        for (int p = 0; p < kTwo<T>; ++p)
                            ov[mat][p] = mma(c == 0 && ks == 0 ? zero4 : ov[mat][p], fr[i & 1][ks], hs[c * KC + ks].t[p]);
                }
                const f32x4 e4 = ld4(decay + k0 + 4 * q);
#pragma unroll
                for (int p = 0; p < kTwo<T>; ++p) {
                    settle(ov[0][p]);
                    if (DELTA) settle(ov[MATS - 1][p]);
                }
                O[kt] = e4 * (kTwo<T> == 2 ? ov[0][0] + ov[0][kTwo<T> - 1] : ov[0][0]);
                if (DELTA) {
                    const f32x4 v = kTwo<T> == 2 ? ov[MATS - 1][0] + ov[MATS - 1][kTwo<T> - 1] : ov[MATS - 1][0];
                    const f32x4 b4 = ld4(betas + (mine ? hw : 0) * kp + k0 + 4 * q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) Rt[kt][e] = e4[e] < 0.f ? 0.f : b4[e] * (xt[kt][e] - e4[e] * v[e]);
                }
            }
        }
        if (CF::STG) {  // the table rows of this wave again, from LDS: the state's products had their registers
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) rs[ks] = kept(DELTA && kind ? x2 : x1, tw, ks);
        }
#pragma unroll 1
        for (int sp = 0; sp <= s; ++sp) {
            const bool own = sp == s;
            const int j0 = sp * kPanel;
            again();
            // the tables are free, and so is x1 (the products with C, or the panel before, are done)
            if (CF::STG && sp == 0 && !own) {
                F8 bn[KH];
                ask_b(0, bn);
                __syncthreads();
                keep_b(bn);
                __syncthreads();
            } else if (s > 0) {
                __syncthreads();
            }
            // ---- this wave's table rows against panel sp ----
            if (tw < nk) {
                const int k = q0 + 16 * tw + l16;
                const u64 path = mask[sp * kp + k];
                const T* bj0 = own ? x2 : x1;
                T* tab = (DELTA && kind ? ttabs : mtabs) + tw * TAB;
                F8 fr[2][KC];
                constexpr int JT = DELTA ? 4 : 2;
                const int jt0 = DELTA ? 0 : 2 * kind;
                auto ask = [&](int i) {
#pragma unroll
                    for (int ks = 0; ks < KC; ++ks)
                        fr[i & 1][ks] = CF::STG ? kept(bj0, jt0 + i / CH, i % CH * KC + ks)
                                                : frag(Bm, a.bs, j0 + 16 * (jt0 + i / CH) + l16, i % CH * KC + ks);
                };
                ask(0);
#pragma unroll
                for (int j = 0; j < JT; ++j) {
                    const int jt = jt0 + j;
                    if (!own || jt < ((tw + 2) & ~1)) {
                        __builtin_amdgcn_sched_barrier(0);
                        f32x4 c = zero4;
#pragma unroll
                        for (int i = 0; i < CH; ++i) {
                            F8(&f)[KC] = fr[(j * CH + i) & 1];
                            together(f);
                            if (j * CH + i + 1 < JT * CH) ask(j * CH + i + 1);
#pragma unroll
                            for (int ks = 0; ks < KC; ++ks)
                                c = mma(c, f[ks], CF::STG ? rs[i * KC + ks] : DELTA ? frag(rows, rows_st, k, i * KC + ks) : frag(Cm, a.cs, k, i * KC + ks));
                        }
                        settle(c);
#pragma unroll
                        for (int hd = 0; hd < 2; ++hd)
                            if (hd < place.nh) {
                                // (no node behind its own is on its path, so the tile past the last is zero of itself; T's
                                // diagonal tile is in its inverse)
                                const float* dh = decays + hd * kp;
                                const double* ch = css + hd * kp;
                                f32x4 v = weigh(dh[k] < 0.f ? 0u : (unsigned)(path >> (16 * jt + 4 * q)) & 15u, ch[k],
                                                ch + j0 + 16 * jt + 4 * q, DELTA && kind ? betas[hd * kp + k] : 1.f, c);
                                if (DELTA && kind && own && jt == tw) v = zero4;
                                put(tab + hd * 4 * TAB, jt >> 1, jt & 1, lane, v);
                            }
                    }
                }
                // head `kind`'s inverses: two tiles each for the waves with the shorter table rows
                if (DELTA && own && tw < 2 && kind < place.nh)
#pragma unroll 1
                    for (int it = tw; it < nk && it <= 3 - tw; it += 3 - 2 * tw) {
                        f32x4 b = zero4;
#pragma unroll
                        for (int i = 0; i < CH; ++i) {
#pragma unroll
                            for (int ks = 0; ks < KC; ++ks)
                                fr[0][ks] = CF::STG ? kept(x2, it, i * KC + ks) : frag(Bm, a.bs, q0 + 16 * it + l16, i * KC + ks);
                            together(fr[0]);
#pragma unroll
                            for (int ks = 0; ks < KC; ++ks) b = mma(b, fr[0][ks], fr[0][ks]);
                        }
                        settle(b);
                        const int n = kind * kp + q0 + 16 * it;
                        const u64 strict = decays[n + l16] < 0.f ? 0 : mask[s * kp + q0 + 16 * it + l16] & ~(1ull << (16 * it + l16));
                        T* inv = reinterpret_cast<T*>(smem + at.inv + (kind * 4 + it) * 1024);
                        const f32x4 t = weigh((unsigned)(strict >> (16 * it + 4 * q)) & 15u, css[n + l16], css + n + 4 * q, betas[n + l16], b);
                        put_inv(inv, lane, inverse16(t, reinterpret_cast<float*>(inv), lane));
                    }
            }
            if (CF::STG && sp + 1 < s) {
                F8 bn[KH];
                ask_b(j0 + kPanel, bn);
                __syncthreads();
                keep_b(bn);  // (read behind the next barrier)
            } else {
                __syncthreads();
            }
            again();
            // ---- panel sp's part of Rt and O ----
            F8 xf[2];
            Op<T> uf[2];
            if constexpr (!DELTA) {
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    xf[f] = own ? pair8(x, xt[2 * f], xt[2 * f + 1])
                                : pair8(x, take_x(xn[2 * f], j0 + 32 * f), take_x(xn[2 * f + 1], j0 + 32 * f + 16));
                if (sp + 1 < s) ask_x(j0 + kPanel, xn);
            } else if (own) {
                const T* inv0 = reinterpret_cast<const T*>(smem + at.inv + (mine ? hw : 0) * 4096);
                f32x4 u[2];
                split(join(zero4, zero4), uf[0]);
                split(join(zero4, zero4), uf[1]);
#pragma unroll
                for (int kt = 0; kt < 4; ++kt)
                    if (kt < nk && mine) {
                        const auto inv = get_inv(inv0 + kt * 1024 / (int)sizeof(T), lane);
                        f32x4 t = zero4;
                        Op<T> to[2];
#pragma unroll
                        for (int f = 0; 2 * f < kt; ++f) to[f] = get(tt + kt * TAB, f, lane);
#pragma unroll
                        for (int f = 0; 2 * f < kt; ++f) {
                            together(to[f]);
                            t = mul(t, to[f], uf[f]);
                        }
                        u[kt & 1] = times_inv(inv, Rt[kt] - t);
                        split(join(u[0], kt & 1 ? u[1] : zero4), uf[kt >> 1]);
                    }
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    if (s == 0) u0[f] = uf[f];
                    if (s == 1) u1[f] = uf[f];
                    if (s == 2) u2[f] = uf[f];
                }
            } else {
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    uf[f] = u0[f];
                    if (sp == 1) uf[f] = u1[f];
                    if (sp == 2) uf[f] = u2[f];
                }
#pragma unroll
                for (int kt = 0; kt < 4; ++kt)
                    if (kt < nk && mine) {
                        Op<T> t0 = get(tt + kt * TAB, 0, lane), t1 = get(tt + kt * TAB, 1, lane);
                        together(t0);
                        together(t1);
                        f32x4 t = mul(mul(zero4, t0, uf[0]), t1, uf[1]);
                        settle(t);
                        Rt[kt] -= t;
                    }
            }
            if (own) {  // the next panel's rows
                __builtin_amdgcn_sched_barrier(0);
                if (CF::STG) ask_own(q0 + kPanel);
                ask_x(q0 + kPanel, xq);
            }
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
                if (kt < nk && mine) {
                    Op<T> m0 = get(mt + kt * TAB, 0, lane), m1 = get(mt + kt * TAB, 1, lane);
                    together(m0);
                    together(m1);
                    if constexpr (DELTA) {
                        O[kt] = mul(O[kt], m0, uf[0]);
                        if (!own || kt >= 2) O[kt] = mul(O[kt], m1, uf[1]);
                    } else {
                        O[kt] = mul(O[kt], m0, xf[0]);
                        if (!own || kt >= 2) O[kt] = mul(O[kt], m1, xf[1]);
                    }
                    settle(O[kt]);
                }
        }
        again();
        // ---- y ----
#pragma unroll
        for (int kt = 0; kt < 4; ++kt)
            if (kt < nk && mine) {
                const int k0 = q0 + 16 * kt;
                const f32x4 e4 = ld4(decay + k0 + 4 * q);
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float o = DELTA ? O[kt][e] : O[kt][e] + D * xt[kt][e];
                    v[e] = e4[e] == -1.f ? 0.f : e4[e] == -2.f ? nan : o;
                }
                if (anybad) {  // a bad x on the node's path
                    unsigned hits = 0;
#pragma unroll 1
                    for (int i = 0; i < 4 * (s + 1); ++i)
                        if (mask[(i >> 2) * kp + k0 + 4 * q + (i & 3)] & badx[(i >> 2) * badp]) hits |= 1u << (i & 3);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (hits >> e & 1 && !(e4[e] < 0.f)) v[e] = nan;
                }
                store_y(y, ys, k0, K, lane, sel, upper, v);
            }
    }
}

// Heads of a group that a work-group takes one after another: the fewest rounds of work-groups (as many at once as LDS
// lets in, up to three a CU), each of which costs its heads and two more for what they share.  One / the rule's / four /
// eight heads: 64 trees of 64 nodes, 80 heads in one group 85 / 68 / 68 / 74 us, the delta rule 131 / 92 / 95 / 109; 8 of
// them 15.7 / 15.5 / 20 / 33; one tree of 8 nodes over 48 heads 9.6 / 9.7 / 9.9 / 15.9.
inline int tree_heads(const Args& a, int slabs, int lds0, int lds_head) {
    const int hg = a.H / a.G;
    int best = 1;
    int64_t least = 0;
    for (int hb = 1; hb <= 8 && hb <= hg; ++hb) {
        const int64_t groups = a.b * a.G * ((hg + hb - 1) / hb) * slabs, fit = 160 * 1024 / (lds0 + hb * lds_head);
        const int64_t at_once = 256 * (fit > 3 ? 3 : fit < 1 ? 1 : fit);
        const int64_t cost = (groups + at_once - 1) / at_once * (hb + 2);
        if (hb == 1 || cost < least) least = cost, best = hb;
    }
    return best;
}

// `groups` work-groups a row.  Rows go in as many launches as a launch's threads take (a row has at most 2^29: nheads *
// headdim is at most 2^24).
template <typename T, typename K>
int launch_rows(K* kernel, const Args& a, int heads, int64_t groups, int threads, size_t lds) {
    if (!delta::lds_limit(kernel, lds)) return 7;
    const int64_t most = kMaxThreads / (groups * threads);
    for (int64_t row = 0; row < a.b; row += most) {
        const int64_t tok = row * a.T;
        Args p = a;
        p.b = a.b - row < most ? a.b - row : most;
        p.x = static_cast<const T*>(a.x) + tok * a.xs;
        p.dt = a.dt + tok * a.H;
        p.B = static_cast<const T*>(a.B) + tok * a.bs;
        p.C = static_cast<const T*>(a.C) + tok * a.cs;
        if (a.beta) p.beta = static_cast<const T*>(a.beta) + tok * a.H;
        p.parents = a.parents + tok;
        p.slots = a.slots + row;
        p.y = static_cast<T*>(a.y) + tok * a.H * a.P;
        kernel<<<(unsigned)(p.b * groups), threads, lds, a.stream>>>(p, heads);
    }
    return hipGetLastError() == hipSuccess ? 0 : 7;
}

template <typename T, int N, bool DELTA, int NK>
int launch_tree(const Args& a) {
    typedef TreeCfg<T, N, DELTA, NK> CF;
    const int cols = a.P < 64 ? a.P / 16 : 4, waves = cols > NK ? cols : NK;
    const int slabs = a.P / (16 * cols), hg = a.H / a.G, hb = tree_heads(a, slabs, CF::C, CF::HEAD);
    return launch_rows<T>(k_tree<T, N, DELTA, NK>, a, hb, (int64_t)a.G * ((hg + hb - 1) / hb) * slabs, 64 * waves, CF::total(hb));
}
template <typename T, int N, bool DELTA>
int run_tree_n(const Args& a) {
    if (a.T <= 16) return launch_tree<T, N, DELTA, 1>(a);
    if (a.T <= 32) return launch_tree<T, N, DELTA, 2>(a);
    if (a.T <= 48) return launch_tree<T, N, DELTA, 3>(a);
    if (a.T <= kPanel) return launch_tree<T, N, DELTA, 4>(a);
    typedef LongCfg<T, N, DELTA> CF;
    // Two heads a work-group where one each would leave CUs a second one and the waves suffice (one / two: 16 lines of
    // 200 nodes above 127 / 85 us, the scan 99 / 61, in float32 628 / 379 and 377 / 213; 16 rows of 65 nodes at dstate 128
    // 44 / 28, the scan 35 / 22; 9 rows of 200 at dstate 256 120 / 79, the scan 93 / 57).
    const int hg = a.H / a.G, heads = a.P <= 64 && hg > 1 && a.b * a.H > 256 ? 2 : 1;
    const size_t lds = (size_t)LongLds((int)a.T, heads, a.P / 16, DELTA, CF::STG ? CF::ROWS : 0).total;
    return launch_rows<T>(k_tree_long<T, N, DELTA>, a, heads, (int64_t)a.G * ((hg + heads - 1) / heads), 512, lds);
}
template <typename T, bool DELTA>
int run_tree_rule(const Args& a) {
    switch (a.N) {
        case 16: return run_tree_n<T, 16, DELTA>(a);
        case 32: return run_tree_n<T, 32, DELTA>(a);
        case 64: return run_tree_n<T, 64, DELTA>(a);
        case 128: return run_tree_n<T, 128, DELTA>(a);
        case 256: return run_tree_n<T, 256, DELTA>(a);
        default: return 3;
    }
}
template <typename T>
int run_tree(const Args& a) { return a.beta ? run_tree_rule<T, true>(a) : run_tree_rule<T, false>(a); }

int tree_bf16(const Args& a);
int tree_f32(const Args& a);

}  // namespace pool
}  // namespace ssd
