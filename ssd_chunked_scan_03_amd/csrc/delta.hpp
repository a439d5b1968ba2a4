// delta.hpp -- the gated delta rule on the scan's operands (x, dt, A, B, C) with a write
// strength beta per token and head:
//
//   r_t = x_t - a_t h_{t-1} B_t      what the decayed state does not yet answer to key B_t
//   h_t = a_t h_{t-1} + beta_t r_t B_t^T,   y_t = h_t C_t,   a_t = exp(dt_t A_h)
//
// Chunks of L = 64 tokens.  With c the cumulative sum of dt A in the chunk, K and Q the
// chunk's B and C rows, G_ij = exp(c_i - c_j) (i >= j), h the state entering the chunk:
//
//   KK = strict_tril(G o K K^T),  M = tril(G o Q K^T)
//   S  = (I + KK diag(beta))^-1 KK                       (strictly lower, one per chunk and head)
//   R  = X - diag(e^c) K h^T,  r = R - S (beta R),  u = beta r
//   Y  = diag(e^c) Q h^T + M u
//   h' = e^{c_L} h + (diag(e^{c_L - c}) u)^T K
//
// r follows from S without a division by beta (r = (I + KK diag(beta))^-1 R and
// (I + KK diag(beta))^-1 = I - S diag(beta)), and the adjoint needs the same S:
//
//   dU = M^T dY + diag(e^{c_L - c}) K dh'^T,  z = dU - S^T (beta dU),  dX = beta z
//   dh = e^{c_L} dh' + (diag(e^c) dY)^T Q - (diag(e^c) dX)^T K
//   dP_ij = G_ij beta_j dY_i . r_j (i >= j),  W_ij = -beta_i G_ij beta_j z_i . r_j (i > j)
//   dQ = diag(e^c) dY h + dP K,  dbeta_i = z_i . r_i
//   dK = dP^T Q + (W + W^T) K + diag(e^{c_L - c} beta) r dh' - diag(e^c) dX h
//   dlog a_t = sum_{i >= t > j} E_ij + sum_{i >= t} F_i + sum_{j < t} D_j + e^{c_L} <dh', h>,
//     E_ij = dP_ij (Q_i . K_j) + W_ij (K_i . K_j),   F_i = e^{c_i} (dY_i . h Q_i - dX_i . h K_i),
//     D_j = e^{c_L - c_j} u_j . dh' K_j
//
// The last sums over everything whose decay holds a_t: pairs of tokens on either side, the
// entering state with a later token, an earlier token with the leaving state, and one state
// with the other.  (It is also sum_{s >= t} (dY_s . Y_s - dX_s . X_s) + <dh', h'>, whose terms
// are of order one however little of a state outlives a token: their difference loses the
// gradient of a strong decay.)
//
// Precision.  One bfloat16 rounding of the state in a product would cost 2e-3 of the float32
// outputs (hT, ddt, dA, dh0), so float32 operands enter the matrix cores as a sum of three
// bfloat16 terms (8 bits each: the whole float32 mantissa): 3 products against an operand
// that is bfloat16 already, the 6 of order <= 2 between two split ones.  Products that only
// reach bfloat16 outputs take fewer terms (noted where).  float32 problems run on the
// float32 matrix cores throughout.
//
// Tiles.  A wave keeps the state of 16 or 32 headdim columns, h^T[n][p], in accumulators.
// The accumulator layout (lane l: rows 4 (l / 16) + e, column l % 16) of two row tiles is a
// matrix-core B operand whose k index runs 16 (e / 4) + 4 (l / 16) + e % 4; with the A
// operand read in that same k order, every product of the chunk feeds the next one from
// registers, and waves never exchange data.
#pragma once

#include <type_traits>

#include "kernels.hpp"

namespace ssd {
namespace delta {

constexpr int L = 64;                 // tokens per chunk
constexpr int kTri = 10;              // 16 x 16 blocks on and below the diagonal of a 64 x 64 table
constexpr int kTab = 2 * kTri * 256;  // floats of one (chunk, head)'s S and M tables
constexpr int kVec = 5 * L;           // floats of its e^c, e^{c_L - c}, beta and c (log2 units, two parts)
// Forward tables of one (chunk, head) as operand fragments (bfloat16, dstate 64 and up): -S
// diag(beta) in three terms, then M diag(beta) in two (one would cost y as much as its own
// rounding wherever M u cancels), [term][fragment][lane][8]; the 10 blocks on and
// below the diagonal fill 5 fragments (frag_at), and beta is folded into their columns and
// into the e^{c_L - c} of vec, so that the walk never reads it.
constexpr int kFragTab = (3 + 2) * 5 * 512;  // bfloat16 elements
// The backward's: -S and M, three terms each, nothing folded.
constexpr int kFragTab2 = (3 + 3) * 5 * 512;
// Behind either, the decay factors of the walk (float32): e^c, e^{c_L - c} (times beta where
// folded), and for the backward beta.
constexpr int kFragVec = 512;  // bfloat16 elements (1 KiB, one transfer)
enum Tab { kPlain, kFold, kBoth };  // tables as float32 blocks, the forward's, the backward's fragments
constexpr int kFrag = 6;              // 16 x 32 operand fragments covering a triangular 64 x 64 table

struct Args {
    Rows rows;
    int64_t T;   // dense: tokens per row; packed: tokens of the axis
    int H, P, N, G, nc;
    int ntab;    // chunks of the table axis (dense b nc, packed kcap)
    const void* x;
    const float* dt;
    const float* A;
    const void* B;
    const void* C;
    const void* beta;
    const float* h0;
    void* y;
    float* hT;
    float* tab;  // [ntab][H][kTab]
    float* vec;  // [ntab][H][kVec]
    // backward
    const void* dy;
    const float* dhT;
    void* dx;
    float* ddt;
    float* dA;
    void* dB;
    void* dC;
    void* dbeta;
    float* dh0;
    void* r;      // [b T][H][P] residuals; bfloat16: in three terms
    void* rlo;
    void* rll;
    void* z;      // [b T][H][P], the same
    void* zlo;
    void* zll;
    float* kh;    // [ntab][H] e^c K h^T, 64 P values as the walks hold them (kh_at)
    void* hin;    // [ntab][H][P][N] state entering each chunk
    short* hlo;   // bfloat16: what hin's rounding left of the float32 state (split_state)
    void* lin;    // [ntab][H][P][N] dh' of each chunk
    float* fq;    // [slices][b H][T] per-slice e^c dY . h Q
    float* fk;    // [slices][b H][T] per-slice e^c dX . h K
    float* dj;    // [slices][b H][T] per-slice D
    float* tot;   // [tots][ntab][H] per-wave e^{c_L} <dh', h> of each chunk
    double* dAp;  // [ntab][H]
    float* part;  // [nsub][2][b T][G][N] partial dK, dQ when a group's heads are shared out
    int slices, tots, nsub;
    int* order;   // packed: [nrows] the rows in the order that the walks start them
    hipStream_t stream;
};

// ---------------------------------------------------------------------------
// float32 operands as sums of matrix-core operands: pairs are converted together (one
// instruction each way), 5.5 operations an element for three terms
// ---------------------------------------------------------------------------
template <typename T> struct Sp;
template <> struct Sp<bf16> { bf16x8 t[3]; };
template <> struct Sp<float> { f32x8 t[1]; };
template <typename T> constexpr int kTerms = std::is_same<T, bf16>::value ? 3 : 1;

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
// two bfloat16, rounded to nearest, in one instruction
__device__ __forceinline__ unsigned cvt2(float a, float b) {
    return __builtin_bit_cast(unsigned, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
template <int NB = 3>
__device__ __forceinline__ void split8(f32x8 v, Sp<bf16>& s) {
    u32x4v o[3];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float a = v[e], b = v[e + 1];
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const unsigned u = cvt2(a, b);
            o[k][e >> 1] = u;
            if (k + 1 < NB) {
                a -= __builtin_bit_cast(float, u << 16);
                b -= __builtin_bit_cast(float, u & 0xffff0000u);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) s.t[k] = __builtin_bit_cast(bf16x8, o[k]);
}
template <int NB = 3>
__device__ __forceinline__ void split8(f32x8 v, Sp<float>& s) { s.t[0] = v; }
template <int NB>
__device__ __forceinline__ void split4(f32x4 v, bf16x4 (&o)[NB]) {
    float a[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int k = 0; k < NB; ++k) {
        const u32x2 u = u32x2{cvt2(a[0], a[1]), cvt2(a[2], a[3])};
        o[k] = __builtin_bit_cast(bf16x4, u);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            a[e] -= __builtin_bit_cast(float, e & 1 ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16);
    }
}

// c += a b, a exact in T, b in its first NB terms
template <int NB, typename T, typename V>
__device__ __forceinline__ f32x4 mma_es(f32x4 c, V a, const Sp<T>& b) {
#pragma unroll
    for (int k = 0; k < (NB < kTerms<T> ? NB : kTerms<T>); ++k) c = mma(c, a, b.t[k]);
    return c;
}
// c += a b, both split: the products whose order is under ORD
template <int ORD, typename T>
__device__ __forceinline__ f32x4 mma_ss(f32x4 c, const Sp<T>& a, const Sp<T>& b) {
#pragma unroll
    for (int i = 0; i < kTerms<T>; ++i)
#pragma unroll
        for (int j = 0; j < kTerms<T>; ++j)
            if (i + j < ORD) c = mma(c, a.t[i], b.t[j]);
    return c;
}
// c += a b over k = 16 in float32 (k index 4 (lane / 16) + e for both operands)
__device__ __forceinline__ f32x4 mma16(f32x4 c, f32x4 a, f32x4 b) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

// A float32 state as a bfloat16 (rounded to nearest) and 16 bits of what that left of its bit
// pattern, halved to fit: the gradient products read the first alone, the decay gradient's
// <dh', h'> both, good to 2^-23.
__device__ __forceinline__ void split_state(f32x8 v, bf16x8& hi, s16x8& lo) {
    u32x4v h, l;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const unsigned u = cvt2(v[e], v[e + 1]);
        const int a = __builtin_bit_cast(int, (float)v[e]) - (int)(u << 16);
        const int b = __builtin_bit_cast(int, (float)v[e + 1]) - (int)(u & 0xffff0000u);
        h[e >> 1] = u;
        l[e >> 1] = ((unsigned)(a >> 1) & 0xffffu) | ((unsigned)(b >> 1) << 16);
    }
    hi = __builtin_bit_cast(bf16x8, h);
    lo = __builtin_bit_cast(s16x8, l);
}
__device__ __forceinline__ float join_state(bf16 hi, short lo) {
    return __builtin_bit_cast(float, ((unsigned)__builtin_bit_cast(unsigned short, hi) << 16) + ((unsigned)(int)lo << 1));
}

// Lane exchanges inside a row of 16 in the ALU (a shuffle is an LDS round trip).
template <int CTRL> __device__ __forceinline__ unsigned lane_turn(unsigned v) {
    return (unsigned)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL> __device__ __forceinline__ float lane_turn(float v) {
    return __builtin_bit_cast(float, lane_turn<CTRL>(__builtin_bit_cast(unsigned, v)));
}
// The value N lanes before, in its row of 16 (zero past the row's start).
template <int N> __device__ __forceinline__ float row_shift(float v) { return lane_turn<0x110 + N>(v); }
// Sum over the 16 lanes of a row, in every lane (rotations by 8, 4, 2, 1).
__device__ __forceinline__ float row_sum16(float v) {
    v += lane_turn<0x128>(v);
    v += lane_turn<0x124>(v);
    v += lane_turn<0x122>(v);
    return v + lane_turn<0x121>(v);
}
// The 4 x 4 transpose of 16-bit elements among 4 neighbouring lanes (lane b, element i <-> lane i,
// element b): accumulator columns (4 tokens of one headdim column per lane) <-> rows (4
// columns of one token per lane), so that x, y and their gradients move 8 bytes a lane.  One
// exchange of halves with lane b ^ 1 (`sel`, quad_sel), one of words with lane b ^ 2.
typedef unsigned u32x2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ unsigned quad_sel(int lane) { return lane & 1 ? 0x03020706u : 0x05040100u; }
__device__ __forceinline__ u32x2v quad_t(u32x2v v, unsigned sel, bool upper) {
    const unsigned a = __builtin_amdgcn_perm(lane_turn<0xB1>((unsigned)v[0]), v[0], sel);
    const unsigned b = __builtin_amdgcn_perm(lane_turn<0xB1>((unsigned)v[1]), v[1], sel);
    const unsigned a2 = lane_turn<0x4E>(a), b2 = lane_turn<0x4E>(b);
    return upper ? u32x2v{b2, b} : u32x2v{a, a2};
}
// A wave's 16 CT headdim columns: lane l16 of column tile ct holds column 4 CT (l16 / 4) + 4 ct +
// l16 % 4 of them, so that after the transpose a lane has 4 CT neighbours of one token.
template <int CT>
__device__ __forceinline__ constexpr int tile_col(int l16, int ct) { return 4 * CT * (l16 >> 2) + 4 * ct + (l16 & 3); }
// Those columns of token tile `it` in a [token][H P] tensor (resource at the chunk's first token,
// rows past its end read as zero and drop stores).  xo: byte offset of this lane's token and
// columns.
template <int CT>
__device__ __forceinline__ int rows_off(int lane, int rsx, int p0) {
    return (4 * (lane >> 4) + (lane & 3)) * rsx + (p0 + 4 * CT * ((lane & 15) >> 2)) * 2;
}
template <int CT>
__device__ __forceinline__ void load_tile(brsrc r, u32x2v (&o)[CT], int xo, int it, int rsx) {
    if constexpr (CT == 2) {
        const u32x4v v = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(r, xo, it * 16 * rsx, 0));
        o[0] = u32x2v{v[0], v[1]};
        o[1] = u32x2v{v[2], v[3]};
    } else {
        o[0] = __builtin_bit_cast(u32x2v, __builtin_amdgcn_raw_buffer_load_b64(r, xo, it * 16 * rsx, 0));
    }
}
template <int CT>
__device__ __forceinline__ void store_tile(brsrc r, const f32x4 (&v)[CT], int xo, int it, int rsx, unsigned sel, bool upper) {
    u32x2v w[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
        w[ct] = quad_t(u32x2v{cvt2(v[ct][0], v[ct][1]), cvt2(v[ct][2], v[ct][3])}, sel, upper);
    if constexpr (CT == 2)
        __builtin_amdgcn_raw_buffer_store_b128(u32x4v{w[0][0], w[0][1], w[1][0], w[1][1]}, r, xo, it * 16 * rsx, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, w[0]), r, xo, it * 16 * rsx, 0);
}
__device__ __forceinline__ f32x4 floats(u32x2v v) {
    return f32x4{__builtin_bit_cast(float, v[0] << 16), __builtin_bit_cast(float, v[0] & 0xffff0000u),
                 __builtin_bit_cast(float, v[1] << 16), __builtin_bit_cast(float, v[1] & 0xffff0000u)};
}
// what rounding to bfloat16 leaves of v
__device__ __forceinline__ f32x4 rest16(f32x4 v) {
    return v - floats(u32x2v{cvt2(v[0], v[1]), cvt2(v[2], v[3])});
}

// Where a wave's lane finds its four tokens of token tile `it`, column tile ct, of a chunk's e^c K
// h^T: `tiles` = the wave's group of 16 CT columns, of P / (16 CT).
template <int CT>
__device__ __forceinline__ int64_t kh_at(int64_t item, int P, int tiles, int it, int ct, int lane) {
    return item * L * P + (int64_t)((tiles * 4 + it) * CT + ct) * 256 + lane * 4;
}

__device__ __forceinline__ f32x8 join(f32x4 a, f32x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// A operand of row `row`, columns k0 + 16 (e / 4) + 4 q + e % 4, of a row-major tile
template <typename T>
__device__ __forceinline__ typename V8<T>::type frag_k(const T* M, int ld, int row, int k0, int q) {
    return join(ld4(M + row * ld + k0 + 4 * q), ld4(M + row * ld + k0 + 16 + 4 * q));
}

__host__ __device__ constexpr int tri(int i, int j) { return i * (i + 1) / 2 + j; }
// fragment of row tile i, 32 columns t of a lower triangular table (t <= i / 2), and of an
// upper triangular one (t >= i / 2)
__host__ __device__ constexpr int frag_lo(int i, int t) { return i < 2 ? i : 2 + (i - 2) * 2 + t; }
__host__ __device__ constexpr int frag_up(int i, int t) { return i < 2 ? i * 2 + t : 4 + (i - 2); }

// element offset, in a table of 5 fragments, of block (i, j)'s four elements of lane 0
__host__ __device__ constexpr int frag_at(int i, int j) {
    return i == 0 ? 0 : i == 2 && j == 2 ? 4 : (i < 3 ? i : 3 + (j >> 1)) * 512 + 4 * (j & 1);
}
// the 16 x 32 fragment of row tile i, columns 32 t on
__device__ __forceinline__ bf16x8 frag_tab5(const bf16* tab, int i, int t, int lane) {
    const bf16x4 z = bf16x4{(bf16)0.f, (bf16)0.f, (bf16)0.f, (bf16)0.f};
    if (i == 0) return join(ld4(tab + lane * 8), z);
    if (i == 2 && t == 1) return join(ld4(tab + lane * 8 + 4), z);
    return ld8(tab + frag_at(i, 2 * t) + lane * 8);
}

// The triangular table `src` (16 x 16 blocks, row-major, as k_delta_prep stores it) by way of 256
// threads' registers into LDS as operand fragments: dst[term][fragment][lane][8].  UP: its
// transpose.  Thread t holds lane t % 64's 4 elements of blocks t / 64, + 4 and + 8 (10 stored
// blocks and the two zero ones that complete fragments).
template <bool UP>
__device__ __forceinline__ void get_tri(const float* __restrict__ src, f32x4 (&v)[3]) {
    const int l = threadIdx.x & 63, l16 = l & 15, q = l >> 4;
#pragma unroll
    for (int u = 0; u < 3; ++u) {
        const int blk = wave_id() + 4 * u;
        v[u] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (blk < kTri) {
            if (UP) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[u][e] = src[blk * 256 + (4 * q + e) * 16 + l16];
            } else {
                v[u] = ld4(src + blk * 256 + l16 * 16 + 4 * q);
            }
        }
    }
}
template <typename T, int NT, bool UP>
__device__ __forceinline__ void put_tri(const f32x4 (&s)[3], T* dst) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int u = 0; u < 3; ++u) {
        const int blk = wave_id() + 4 * u;
        int i, j;  // block row, column
        if (blk < kTri) {
            i = blk < 1 ? 0 : blk < 3 ? 1 : blk < 6 ? 2 : 3;
            j = blk - tri(i, 0);
        } else {
            i = blk == kTri ? 0 : 2;
            j = i + 1;
        }
        f32x4 v = s[u];
        const int f = UP ? frag_up(j, i >> 1) : frag_lo(i, j >> 1);
        T* d = dst + f * 512 + l * 8 + 4 * ((UP ? i : j) & 1);
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            typename V4<T>::type o;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[e] = from_f<T>(v[e]);
                v[e] -= to_f(o[e]);
            }
            st4(d + k * kFrag * 512, o);
        }
    }
}
template <typename T, int NT>
__device__ __forceinline__ Sp<T> frag_tab(const T* tab, int f, int lane) {
    Sp<T> s;
#pragma unroll
    for (int k = 0; k < NT; ++k) s.t[k] = ld8(tab + (k * kFrag + f) * 512 + lane * 8);
    return s;
}

// Every wave's LDS reads are done, or (LOADS) its transfers have landed; transfers that no
// wave reads yet stay in flight (a __syncthreads would wait for them all).
__device__ __forceinline__ void wave_meet(bool loads) {
    if (loads) __builtin_amdgcn_s_waitcnt(0xF70);  // vmcnt(0)
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// rows [0, n) x cols [0, w) of src (row stride ss) into dst (row stride ds), rows [n, 64) and
// columns [w, wpad) zero; w a multiple of 8
template <typename T>
__device__ __forceinline__ void stage_rows(const T* __restrict__ src, int64_t ss, T* dst, int ds, int n, int w,
                                           int wpad, int tid, int nthr, int nrows = L) {
    const int per = wpad >> 3;
    for (int p = tid; p < nrows * per; p += nthr) {
        const int row = p / per, col = (p - row * per) << 3;
        typename V8<T>::type v = zero8<T>();
        if (row < n && col < w) v = ld8(src + row * ss + col);
        st8(dst + row * ds + col, v);
    }
}
template <typename T>
__device__ __forceinline__ void store_rows(T* __restrict__ dst, int64_t ds, const T* src, int ss, int n, int w,
                                           int tid, int nthr) {
    const int per = w >> 3;
    for (int p = tid; p < n * per; p += nthr) {
        const int row = p / per, col = (p - row * per) << 3;
        st8(dst + row * ds + col, ld8(src + row * ss + col));
    }
}

// Blocks k, k + 8, k + 16, ... run on one XCD: block k of n takes the item that gives each XCD a
// contiguous range of them, so that neighbours share what they read through one L2.
__device__ __forceinline__ unsigned xcd_range(unsigned k, unsigned n) {
    const unsigned x = k & 7, r = n & 7;
    return x * (n >> 3) + (x < r ? x : r) + (k >> 3);
}
// The (head, slice) items of the walks, in ranges within each row: the slices of a head share
// its tables, the heads of a group its keys.  Packed rows run in `order`, longest first: a
// long row that starts last would be walked alone.
struct Item {
    int bh, sl;
};
__device__ __forceinline__ Item xcd_item(unsigned k, int H, int nsl, const int* order) {
    const unsigned n = (unsigned)H * nsl, it = xcd_range(k % n, n);
    const int r = (int)(k / n), row = order ? order[r] : r;
    return Item{row * H + (int)(it / nsl), (int)(it % nsl)};
}
// That order, by one wave: rows by the power of two below their chunks, descending (one pass
// for the powers there are, one for each; past 1024 rows, where no row is much of the whole, as
// they come).
__device__ __forceinline__ void order_rows(const Rows& rows, int* order, int lane) {
    const int n = rows.nrows;
    if (n > 1024) {
        for (int r = lane; r < n; r += 64) order[r] = r;
        return;
    }
    auto key = [&](int r) { return 32 - __clz(rows.nchunks(r)); };
    unsigned there = 0;
    for (int r = lane; r < n; r += 64) there |= 1u << key(r);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) there |= (unsigned)__shfl_xor((int)there, off, 64);
    int at = 0;
    for (int k = 31; k >= 0; --k) {
        if (!(there >> k & 1)) continue;
        for (int r0 = 0; r0 < n; r0 += 64) {
            const int r = r0 + lane;
            const bool mine = r < n && key(r) == k;
            const uint64_t m = __ballot(mine);
            if (mine) order[at + __popcll(m & ((1ull << lane) - 1))] = r;
            at += __popcll(m);
        }
    }
}

// ---------------------------------------------------------------------------
// k_delta_prep: S and M of a (chunk, head), and the chunk's decay factors; one wave per item,
// no barriers.  A wave takes one (chunk, group) and `heads` of its heads: K K^T and Q K^T once,
// on the matrix cores straight from global rows, kept in accumulators in the orientations
// the steps below read; then per head the decays and S by blocked substitution in float32:
// the four diagonal blocks S_ii side by side (16 lanes each, a lane per column, rows in
// order through LDS), and below the diagonal, transposed so that every product's result is
// the next one's operand and leaves in the order the walks load,
//   Z^T = KK_ij^T - sum_{j < k <= i} KK_kj^T (beta_k S_ik^T),   S_ij^T = Z^T - S_jj^T (beta_j Z^T).
// (The product form (I - X)(I + X^2)(I + X^4)... of the inverse needs no substitution but loses
// four digits where keys repeat.)  Decay sums are float64 and kept in two float32 parts, so
// a strongly decayed chunk keeps the exact ratio of neighbouring tokens.
// TAB: float32 blocks, or the operand fragments that the forward's or the backward's
// fragment walks read.
// Bound by the tables' way to memory: 26 KB per (chunk, head) forward (bfloat16, dstate 64 and
// up), 31 KB backward; 40960 of them (8 rows of 4096 tokens, 80 heads) in 216 to 279 us (the clock
// gives way), 4.9 to 3.8 TB/s.
// Small problems wait for the substitution's chain instead (16 us).
// ---------------------------------------------------------------------------
struct PrepLds {
    float chi[L], clo[L], bet[L];
    float d[4][16][20];  // the diagonal blocks of KK, then of S
};

template <typename T, int N, Tab TAB>
__global__ __launch_bounds__(256, 2) void k_delta_prep(Args a, int heads) {
    constexpr bool FRAG = TAB != kPlain, FOLD = TAB == kFold;
    constexpr double LOG2E = 1.4426950408889634;
    __shared__ __attribute__((aligned(16))) PrepLds lds[4];
    const int lane = threadIdx.x & 63, w = wave_id(), l16 = lane & 15, q = lane >> 4;
    PrepLds& m = lds[w];
    const int H = a.H, G = a.G, Hg = H / G, nhb = (Hg + heads - 1) / heads;
    if (a.order && blockIdx.x == 0 && w == 0) order_rows(a.rows, a.order, lane);
    const int64_t id = (int64_t)blockIdx.x * 4 + w;
    const int hb = (int)(id % nhb), g = (int)(id / nhb % G);
    const int64_t kk = id / nhb / G;
    if (kk >= a.rows.total_chunks()) return;
    const int row = a.rows.row_of((int)kk), c = (int)kk - a.rows.kbase(row);
    const int64_t t0 = a.rows.tok0(row) + (int64_t)c * L;
    const int n = (int)min((int64_t)L, a.rows.len(row) - (int64_t)c * L);

    // off-diagonal pairs (i, j), i > j, in order (1,0) (2,0) (2,1) (3,0) (3,1) (3,2)
    const T* Kg = static_cast<const T*>(a.B) + (t0 * G + g) * N;
    const T* Qg = static_cast<const T*>(a.C) + (t0 * G + g) * N;
    const int64_t rs = (int64_t)G * N;
    f32x4 k1[6], k2[6], kd[4], qk[kTri];  // [i][j] (rows i), [j][i], [i][i], [j][i] of Q K^T
#pragma unroll
    for (int v = 0; v < 6; ++v) k1[v] = k2[v] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < 4; ++v) kd[v] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kTri; ++v) qk[v] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < (N + 31) / 32; ++ks) {
        const int col = ks * 32 + 8 * q;
        const bool in = N >= 32 || col < N;
        const int cc = in ? col : 0;
        typename V8<T>::type kf[4], qf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 16 + l16, rc = r < n ? r : n - 1;
            kf[i] = sel8(in && r < n, ld8(Kg + rc * rs + cc));
            qf[i] = sel8(in && r < n, ld8(Qg + rc * rs + cc));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            kd[i] = mma(kd[i], kf[i], kf[i]);
#pragma unroll
            for (int j = 0; j <= i; ++j) {
                qk[tri(i, j)] = mma(qk[tri(i, j)], kf[j], qf[i]);
                if (j < i) {
                    k1[tri(i - 1, j)] = mma(k1[tri(i - 1, j)], kf[i], kf[j]);
                    k2[tri(i - 1, j)] = mma(k2[tri(i - 1, j)], kf[j], kf[i]);
                }
            }
        }
    }
    const int h0 = g * Hg + hb * heads, h1 = min(g * Hg + Hg, h0 + heads);
    for (int h = h0; h < h1; ++h) {
        const int64_t e0 = kk * H + h;
        float* St = a.tab + e0 * kTab;
        T* Sg = reinterpret_cast<T*>(a.tab) + e0 * ((FOLD ? kFragTab : kFragTab2) + kFragVec);
        T* Mg = Sg + 3 * 5 * 512;
        {
            const bool on = lane < n;
            const int64_t t = t0 + (on ? lane : 0);
            double v = on ? (double)a.dt[t * H + h] * (double)a.A[h] * LOG2E : 0.0;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const double o = __shfl_up(v, off, 64);
                if (lane >= off) v += o;
            }
            const float hi = (float)v, lo = (float)(v - (double)hi);
            const float b = on ? to_f(static_cast<const T*>(a.beta)[t * H + h]) : 0.f;
            const float ew = exp2f_fast((float)(__shfl(v, 63, 64) - v));
            const float ec = exp2f_fast(hi);
            if (FRAG) {
                float* fv = reinterpret_cast<float*>(Sg + (FOLD ? kFragTab : kFragTab2));
                fv[lane] = ec;
                fv[L + lane] = FOLD ? ew * b : ew;
                if (!FOLD) fv[2 * L + lane] = b;
            }
            if (!FOLD) {
                float* vec = a.vec + e0 * kVec;
                vec[lane] = ec;
                vec[L + lane] = ew;
                if (a.ddt) {  // (the backward's)
                    vec[2 * L + lane] = b;
                    vec[3 * L + lane] = hi;
                    vec[4 * L + lane] = lo;
                }
            }
            m.bet[lane] = b;
            m.chi[lane] = hi;
            m.clo[lane] = lo;
        }
        __builtin_amdgcn_wave_barrier();
        f32x4 ch[4], cl[4], bt[4];  // of this lane's rows 4q + e
        float sh[4], sl[4];         // of this lane's column l16
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ch[i] = ld4(m.chi + i * 16 + 4 * q);
            cl[i] = ld4(m.clo + i * 16 + 4 * q);
            bt[i] = ld4(m.bet + i * 16 + 4 * q);
            sh[i] = m.chi[i * 16 + l16];
            sl[i] = m.clo[i * 16 + l16];
        }
        // fragment f of a table from its two blocks' elements (this lane: row l16, columns 4q + e), in
        // TERMS terms: whole 16-byte pieces (halves apart cost 1% of the layer forward).  `first`
        // and `prev` hold a block for its partner (frag_at).
        f32x4 first = f32x4{0.f, 0.f, 0.f, 0.f}, prev = first;
        auto frags = [&](T* dst, int f, f32x4 lo, f32x4 hi, auto terms) {
            Sp<T> sp;
            if constexpr (FRAG) {
                split8<decltype(terms)::value>(join(lo, hi), sp);
#pragma unroll
                for (int k = 0; k < decltype(terms)::value; ++k)  // (past the caches: 2% of the layer forward)
                    __builtin_nontemporal_store(__builtin_bit_cast(u32x4v, sp.t[k]),
                                                reinterpret_cast<u32x4v*>(dst + (k * 5 + f) * 512 + lane * 8));
            }
        };
        auto put = [&](int i, int j, f32x4 v) {  // S_ij, j downward
            if (FRAG) {
                v = FOLD ? v * -bt[j] : -v;
                const std::integral_constant<int, 3> three;
                if (i == 0) first = v;
                else if (i == 2 && j == 2) frags(Sg, 0, first, v, three);
                else if (j & 1) prev = v;
                else frags(Sg, i < 3 ? i : 3 + (j >> 1), v, prev, three);
            } else {
                st4(St + tri(i, j) * 256 + l16 * 16 + 4 * q, v);
            }
        };
        // M, and the diagonal blocks of KK
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j <= i; ++j) {
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float gam = exp2f_fast((sh[i] - ch[j][e]) + (sl[i] - cl[j][e]));
                    v[e] = i > j || l16 >= 4 * q + e ? qk[tri(i, j)][e] * gam : 0.f;
                }
                if (FRAG) {
                    if (FOLD) v *= bt[j];
                    const std::integral_constant<int, FOLD ? 2 : 3> terms;
                    if (i == 0) first = v;
                    else if (i == 2 && j == 2) frags(Mg, 0, first, v, terms);
                    else if (!(j & 1)) prev = v;
                    else frags(Mg, i < 3 ? i : 3 + (j >> 1), prev, v, terms);
                } else {
                    st4(St + (kTri + tri(i, j)) * 256 + l16 * 16 + 4 * q, v);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float gam = exp2f_fast((ch[i][e] - sh[i]) + (cl[i][e] - sl[i]));
                m.d[i][4 * q + e][l16] = 4 * q + e > l16 ? kd[i][e] * gam : 0.f;
            }
        }
        __builtin_amdgcn_wave_barrier();
        {  // S_qq: column l16, rows in order
            float s[16], bs[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float v = m.d[q][i][l16];
#pragma unroll
                for (int k4 = 0; k4 < i; k4 += 4) {
                    const f32x4 kr = ld4(&m.d[q][i][k4]);
#pragma unroll
                    for (int k = k4; k < k4 + 4 && k < i; ++k) v -= kr[k - k4] * bs[k];
                }
                s[i] = v;
                bs[i] = m.bet[q * 16 + i] * v;
            }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < 16; ++i) m.d[q][i][l16] = s[i];
        }
        __builtin_amdgcn_wave_barrier();
        f32x4 sd[4];  // S_jj^T as an A operand: S_jj[4q + e][l16]
#pragma unroll
        for (int j = 0; j < 3; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sd[j][e] = m.d[j][4 * q + e][l16];
        f32x4 b1[6];  // KK_kj^T as A operands
#pragma unroll
        for (int k = 1; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < k; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    b1[tri(k - 1, j)][e] =
                        k1[tri(k - 1, j)][e] * exp2f_fast((ch[k][e] - sh[j]) + (cl[k][e] - sl[j]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4 st[4];  // beta_k S_ik^T
            f32x4 v = ld4(&m.d[i][l16][4 * q]);
            put(i, i, v);
            st[i] = v * bt[i];
#pragma unroll
            for (int j = i - 1; j >= 0; --j) {
                f32x4 zn = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = j + 1; k <= i; ++k) zn = mma16(zn, b1[tri(k - 1, j)], st[k]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = k2[tri(i - 1, j)][e] * exp2f_fast((sh[i] - ch[j][e]) + (sl[i] - cl[j][e])) - zn[e];
                v -= mma16(f32x4{0.f, 0.f, 0.f, 0.f}, sd[j], v * bt[j]);
                put(i, j, v);
                st[j] = v * bt[j];
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// ---------------------------------------------------------------------------
// LDS of the chunk walks (bytes).  Where the K and Q tiles do not fit together (float32 at
// dstate 256) they take turns in one.
// ---------------------------------------------------------------------------
template <typename T, int N>
struct Cfg {
    static constexpr int NP = N < 32 ? 32 : N;      // key columns, padded to a matrix-core k step
    static constexpr int LDK = NP + 8;
    static constexpr bool SHARE = sizeof(T) == 4 && N == 256;
    static constexpr int KT = L * LDK;              // elements of one K / Q tile
    static constexpr int NT = kTerms<T>;
    static constexpr int ldx(int sw) { return sw + 8; }
    static size_t walk_bytes(int sw, int mterms, int xtiles) {
        return (size_t)((SHARE ? 1 : 2) * KT + (NT + mterms) * kFrag * 512 + xtiles * L * ldx(sw)) * sizeof(T) +
               (size_t)(3 * L + 8 * L) * 4;
    }
};

// A chunk's inputs on their way from memory to LDS, in 256 threads' registers: K and Q (dstate
// 256 in float32, where one buffer holds both in turn: the one that is read first, Q in the
// forward walk, K in the adjoint one), x (the adjoint walk: r), dY, the tables of S and M (MT = 0:
// not M) and the factors.
template <typename T, int N, int CT, int MT, bool UP>
struct Staged {
    typedef Cfg<T, N> CF;
    typedef typename V8<T>::type V;
    static constexpr int NK = CF::NP / 32, NX = 2 * CT;  // 8-element pieces per thread
    static constexpr bool K = UP || !CF::SHARE, Q = !UP || !CF::SHARE;
    V k[K ? NK : 1], q[Q ? NK : 1], x[NX], y[NX];
    f32x4 s[3], m[MT ? 3 : 1];
    float f[3];
    template <int C>
    static __device__ __forceinline__ void get(const T* src, int64_t ss, int n, int w, int wpad, V (&v)[C]) {
        const int per = wpad >> 3;
#pragma unroll
        for (int u = 0; u < C; ++u) {
            const int p = (int)threadIdx.x + u * 256, row = p / per, col = (p - row * per) << 3;
            v[u] = zero8<T>();
            if (row < n && col < w) v[u] = ld8(src + row * ss + col);
        }
    }
    template <int C>
    static __device__ __forceinline__ void set(T* dst, int ds, int wpad, const V (&v)[C]) {
        const int per = wpad >> 3;
#pragma unroll
        for (int u = 0; u < C; ++u) {
            const int p = (int)threadIdx.x + u * 256, row = p / per, col = (p - row * per) << 3;
            if (row < L) st8(dst + row * ds + col, v[u]);
        }
    }
    __device__ __forceinline__ void load(const Args& a, int row, int h, int c, int p0, int SW, bool dy) {
        const int H = a.H, G = a.G, P = a.P, g = h / (H / G), t = threadIdx.x;
        const int64_t t0 = a.rows.tok0(row) + (int64_t)c * L, e = (int64_t)(a.rows.kbase(row) + c) * H + h;
        const int n = (int)min((int64_t)L, a.rows.len(row) - (int64_t)c * L);
        if (K) get(static_cast<const T*>(a.B) + (t0 * G + g) * N, (int64_t)G * N, n, N, CF::NP, k);
        if (Q) get(static_cast<const T*>(a.C) + (t0 * G + g) * N, (int64_t)G * N, n, N, CF::NP, q);
        get(static_cast<const T*>(UP ? a.r : a.x) + (t0 * H + h) * P + p0, (int64_t)H * P, n, SW, SW, x);
        if (dy) get(static_cast<const T*>(a.dy) + (t0 * H + h) * P + p0, (int64_t)H * P, n, SW, SW, y);
        get_tri<UP>(a.tab + e * kTab, s);
        if constexpr (MT > 0) get_tri<UP>(a.tab + e * kTab + kTri * 256, m);
        if (t < L) {
            f[0] = a.vec[e * kVec + t];
            f[1] = a.vec[e * kVec + L + t];
            f[2] = t < n ? to_f(static_cast<const T*>(a.beta)[(t0 + t) * H + h]) : 0.f;
        }
    }
    __device__ __forceinline__ void put(T* Ks, T* Qs, T* Xs, T* Ys, T* Sf, T* Mf, float* factors, int SW, bool dy) const {
        const int t = threadIdx.x;
        if (K) set(Ks, CF::LDK, CF::NP, k);
        if (Q) set(Qs, CF::LDK, CF::NP, q);
        set(Xs, CF::ldx(SW), SW, x);
        if (dy) set(Ys, CF::ldx(SW), SW, y);
        put_tri<T, CF::NT, UP>(s, Sf);
        if constexpr (MT > 0) put_tri<T, MT, UP>(m, Mf);
        if (t < L)
#pragma unroll
            for (int i = 0; i < 3; ++i) factors[i * L + t] = f[i];
    }
};

// ---------------------------------------------------------------------------
// k_delta: the chunks of one (row, head) and a slice of 16 W headdim columns, in order (W waves, each
// one column tile: with two, bfloat16 at dstate 32, 512 heads of 64 and 512 tokens take 140 us
// forward against 82 and 718 us backward against 632; no exchange between waves).  All 256 threads stage; a
// chunk's inputs are asked for while the chunk before is computed and wait in registers.  SAVE = false writes y and
// hT.  SAVE = true is the backward's first walk: it writes the residuals r, the state
// entering every chunk, e^c K h^T and the per-token e^c dY . h Q (all terms) instead.
// ---------------------------------------------------------------------------
template <typename T, int N, bool SAVE>
__global__ __launch_bounds__(256) void k_delta(Args a, int waves) {
    typedef Cfg<T, N> CF;
    constexpr int CT = 1;
    constexpr int NP = CF::NP, LDK = CF::LDK, NTL = N / 16, KS = NP / 32, NT = CF::NT;
    constexpr int MT = SAVE ? 0 : NT == 1 ? 1 : 2;  // terms of M (y is rounded to the problem dtype)
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), l16 = lane & 15, q = lane >> 4;
    const int H = a.H, G = a.G, P = a.P;
    const int SW = 16 * CT * waves, ldx = CF::ldx(SW);
    T* Ks = reinterpret_cast<T*>(smem);
    T* Qs = CF::SHARE ? Ks : Ks + CF::KT;
    T* Sf = Qs + CF::KT;
    T* Mf = Sf + NT * kFrag * 512;
    T* Xs = Mf + MT * kFrag * 512;
    T* Ys = Xs + L * ldx;  // SAVE: dY rows
    float* ecs = reinterpret_cast<float*>(Ys + (SAVE ? L * ldx : 0));
    float* ews = ecs + L;
    float* bts = ews + L;
    float* dots = bts + L;  // SAVE: [wave][token]

    const int nsl = P / SW, BH = a.rows.nrows * H;
    const Item it0 = xcd_item(blockIdx.x, H, nsl, a.order);
    const int sl = it0.sl;
    const int64_t bh = it0.bh;
    const int h = (int)(bh % H), row = (int)(bh / H), g = h / (H / G);
    const int64_t Tn = a.rows.len(row), tok0 = a.rows.tok0(row);
    const int nc = a.rows.nchunks(row), kb0 = a.rows.kbase(row);
    const int p0 = sl * SW, pw = w * 16 * CT;  // first column of the slice, of this wave in it
    const bool on = w < waves;                 // the others stage only

    f32x4 acc[NTL][CT];  // h^T: row n = 16 t + 4q + e, column p
#pragma unroll
    for (int t = 0; t < NTL; ++t)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
            acc[t][ct] = a.h0 && on ? ld4(a.h0 + (bh * P + p0 + pw + ct * 16 + l16) * N + t * 16 + 4 * q)
                              : f32x4{0.f, 0.f, 0.f, 0.f};

    Staged<T, N, CT, MT, false> in;
    if (nc > 0) in.load(a, row, h, 0, p0, SW, SAVE);
    for (int c = 0; c < nc; ++c) {
        const int64_t t0 = tok0 + (int64_t)c * L;
        const int n = (int)min((int64_t)L, Tn - (int64_t)c * L);
        const int64_t e = (int64_t)(kb0 + c) * H + h;
        wave_meet(false);  // the previous chunk's tiles are no longer read
        in.put(Ks, Qs, Xs, Ys, Sf, Mf, ecs, SW, SAVE);
        wave_meet(false);
        if (c + 1 < nc) in.load(a, row, h, c + 1, p0, SW, SAVE);
        if (SAVE && on) {
            const int64_t ho = (e * P + p0 + pw) * N;
#pragma unroll
            for (int t = 0; t < NTL; ++t)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const int64_t o = ho + (ct * 16 + l16) * N + t * 16 + 4 * q;
                    if constexpr (std::is_same<T, bf16>::value) {
                        bf16x8 hi;
                        s16x8 lo;
                        split_state(join(acc[t][ct], acc[t][ct]), hi, lo);
                        st4(static_cast<T*>(a.hin) + o, __builtin_shufflevector(hi, hi, 0, 1, 2, 3));
                        *reinterpret_cast<s16x4*>(a.hlo + o) = __builtin_shufflevector(lo, lo, 0, 1, 2, 3);
                    } else {
                        st4(static_cast<T*>(a.hin) + o, acc[t][ct]);
                    }
                }
        }

        // K h^T and Q h^T (Q: two terms are enough for a bfloat16 y)
        f32x4 v[4][CT], yq[4][CT];
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) v[it][ct] = yq[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto state_products = [&](const T* tile, f32x4(&o)[4][CT], auto nb) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                Sp<T> hs[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    split8(join(acc[2 * ks][ct], 2 * ks + 1 < NTL ? acc[2 * ks + 1 < NTL ? 2 * ks + 1 : 0][ct]
                                                                  : f32x4{0.f, 0.f, 0.f, 0.f}),
                           hs[ct]);
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    const auto fr = frag_k(tile, LDK, it * 16 + l16, ks * 32, q);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) o[it][ct] = mma_es<decltype(nb)::value>(o[it][ct], fr, hs[ct]);
                }
            }
        };
        if (on) state_products(Qs, yq, std::integral_constant<int, SAVE ? 3 : 2>());
        if (CF::SHARE) {
            wave_meet(false);
            stage_rows(static_cast<const T*>(a.B) + (t0 * G + g) * N, (int64_t)G * N, Ks, LDK, n, N, NP, tid, 256);
            wave_meet(false);
        }
        if (on) {
        state_products(Ks, v, std::integral_constant<int, 3>());

        // R, then r = R - S (beta R)
        Sp<T> b2[2][CT];
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = it * 16 + 4 * q + i;
                    v[it][ct][i] *= ecs[t];
                }
        if (SAVE) {
#pragma unroll
            for (int it = 0; it < 4; ++it)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) st4(a.kh + kh_at<CT>(e, P, (p0 + pw) / (16 * CT), it, ct, lane), v[it][ct]);
        }
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[it][ct][i] = to_f(Xs[(it * 16 + 4 * q + i) * ldx + pw + ct * 16 + l16]) - v[it][ct][i];
        auto scaled = [&](const float* s, bool two) {  // s_t v_t as operands
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    f32x4 lo = v[2 * t][ct], hi = v[2 * t + 1][ct];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r0 = 32 * t + 4 * q + i;
                        lo[i] *= two ? s[r0] * bts[r0] : s[r0];
                        hi[i] *= two ? s[r0 + 16] * bts[r0 + 16] : s[r0 + 16];
                    }
                    split8(join(lo, hi), b2[t][ct]);
                }
        };
        scaled(bts, false);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            f32x4 d[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) d[ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t <= it / 2; ++t) {
                const Sp<T> sf = frag_tab<T, NT>(Sf, frag_lo(it, t), lane);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) d[ct] = mma_ss<3>(d[ct], sf, b2[t][ct]);
            }
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) v[it][ct] -= d[ct];
        }
        // Y = e^c Q h^T + M u
        if (!SAVE) scaled(bts, false);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i) yq[it][ct][i] *= ecs[it * 16 + 4 * q + i];
            if constexpr (!SAVE) {
#pragma unroll
                for (int t = 0; t <= it / 2; ++t) {
                    const Sp<T> mf = frag_tab<T, MT>(Mf, frag_lo(it, t), lane);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) yq[it][ct] = mma_ss<2>(yq[it][ct], mf, b2[t][ct]);
                }
            }
        }
        // h' = e^{c_L} h + K^T (e^{c_L - c} u)
        scaled(ews, true);
        const float el = ecs[L - 1];
#pragma unroll
        for (int t = 0; t < NTL; ++t) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) acc[t][ct] *= el;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const auto kf = frag_rows_split(Ks, LDK, ks * 32 + 4 * q, ks * 32 + 16 + 4 * q, t * 16, lane);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) acc[t][ct] = mma_es<3>(acc[t][ct], kf, b2[ks][ct]);
            }
        }
        // out through the (own columns of the) x tile: y, or r and the sums with dY
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = it * 16 + 4 * q + i;
                float dot = 0.f;
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    T* o = Xs + t * ldx + pw + ct * 16 + l16;
                    if (SAVE) {
                        T* o2 = Ys + t * ldx + pw + ct * 16 + l16;
                        dot += to_f(*o2) * yq[it][ct][i];
                        *o = from_f<T>(v[it][ct][i]);
                        const float rest = v[it][ct][i] - to_f(*o);
                        *o2 = from_f<T>(rest);
                        if (NT > 1 && t < n)
                            static_cast<T*>(a.rll)[((t0 + t) * H + h) * P + p0 + pw + ct * 16 + l16] =
                                from_f<T>(rest - to_f(*o2));
                    } else {
                        *o = from_f<T>(yq[it][ct][i]);
                    }
                }
                if (SAVE) {
                    dot = row_sum16(dot);
                    if (l16 == 0) dots[w * L + t] = dot;
                }
            }
        }
        wave_meet(false);
        store_rows(static_cast<T*>(SAVE ? a.r : a.y) + (t0 * H + h) * P + p0, (int64_t)H * P, Xs, ldx, n, SW, tid,
                   256);
        if (SAVE) {
            if (NT > 1)
                store_rows(static_cast<T*>(a.rlo) + (t0 * H + h) * P + p0, (int64_t)H * P, Ys, ldx, n, SW, tid, 256);
            for (int t = tid; t < n; t += 256) {
                float s = 0.f;
                for (int k2 = 0; k2 < waves; ++k2) s += dots[k2 * L + t];
                a.fq[((int64_t)sl * BH + bh) * a.T + (int64_t)c * L + t] = s;
            }
        }
    }
    if (!SAVE && a.hT && on) {
#pragma unroll
        for (int t = 0; t < NTL; ++t)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
                st4(a.hT + (bh * P + p0 + pw + ct * 16 + l16) * N + t * 16 + 4 * q, acc[t][ct]);
    }
}

// ---------------------------------------------------------------------------
// k_delta_dma: the forward walk for bfloat16 at dstate 64 and up, every tile fetched straight into
// LDS while the chunk before computes.  Q is refilled once Q h^T is done, the tables once M u
// is done; K, read first and last in a chunk, has two buffers (KB = 2), or one (KB = 1) where
// three work-groups per CU cover the wait; x goes to registers a chunk ahead, and y leaves
// from them.  LDS tiles are unpadded (the transfer writes 16 bytes per lane in order); a row's
// 16-byte pieces are exchanged by the row's low bits, so that the 16 rows of a fragment lie in
// different banks.  Every buffer is an array of its own
// and the two K buffers are named at compile time (chunks in pairs), so the compiler knows
// which reads a transfer in flight does not concern and does not wait for it there.
// Bound by issue and the tables: 8 rows of 4096 tokens, 80 heads of 64, dstate 128, one group, take
// 0.64 to 0.79 ms (the clock gives way); the matrix cores are busy for 46% of the cycles, and other
// vector instructions, most of them the splitting into terms, issue in 41%; x and y alone would take
// 0.13 ms, with the tables 0.34.
// ---------------------------------------------------------------------------
template <int N>
struct Dma {
    static constexpr int PIECES = N / 8;                              // 16-byte pieces of a row
    static constexpr int SWZ = PIECES < 16 ? PIECES - 1 : 15;
    static constexpr int TILE = L * N;                                // elements
};
typedef __attribute__((address_space(3))) void lds_void;

// one wave's share of a 64 x N tile (row stride rs bytes, rows past the resource zero)
template <int N>
__device__ __forceinline__ void dma_tile(brsrc r, bf16* dst, int rs, int w, int nw, int lane) {
    constexpr int RPI = 512 / N, PC = Dma<N>::PIECES;
    for (int m = w; m < L / RPI; m += nw) {
        const int row = m * RPI + lane / PC, j = (lane % PC) ^ (row & Dma<N>::SWZ);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(dst + m * 512), 16, row * rs + j * 16, 0, 0, 0);
    }
}
// `n16` KiB-sized runs of contiguous bytes
__device__ __forceinline__ void dma_run(brsrc r, char* dst, int runs, int w, int nw, int lane) {
    for (int m = w; m < runs; m += nw)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(dst + m * 1024), 16, m * 1024 + lane * 16, 0, 0, 0);
}

template <int N, int KB, int OCC>
__global__ __launch_bounds__(256, OCC) void k_delta_dma(Args a) {
    constexpr int CT = 1, NTL = N / 16, KS = N / 32, TILE = Dma<N>::TILE, SWZ = Dma<N>::SWZ;
    __shared__ __attribute__((aligned(16))) bf16 K0[TILE];
    __shared__ __attribute__((aligned(16))) bf16 K1[KB == 2 ? TILE : 8];
    __shared__ __attribute__((aligned(16))) bf16 Qs[TILE];
    __shared__ __attribute__((aligned(16))) bf16 Sf[kFragTab];  // -S beta in three terms, then M beta in two
    __shared__ __attribute__((aligned(16))) float Vs[2 * L];    // e^c, beta e^{c_L - c}
    const bf16* Mf = Sf + 3 * 5 * 512;
    const int tid = threadIdx.x, nw = blockDim.x >> 6, lane = tid & 63, w = wave_id(), l16 = lane & 15, q = lane >> 4;
    const int H = a.H, G = a.G, P = a.P;
    const int SW = 16 * CT * nw, nsl = P / SW;
    const Item it0 = xcd_item(blockIdx.x, H, nsl, a.order);
    const int sl = it0.sl, bh = it0.bh;
    const int h = bh % H, row = bh / H, g = h / (H / G);
    const int64_t Tn = a.rows.len(row), tok0 = a.rows.tok0(row);
    const int nc = a.rows.nchunks(row), kb0 = a.rows.kbase(row);
    const int p0 = sl * SW + w * 16 * CT;  // this wave's first column

    // h^T: row 4q + e of tile t is n = 32 (t / 2) + 8q + 4 (t % 2) + e, so that a pair of tiles is
    // the operand whose other side reads 8 consecutive columns of K or Q
    f32x4 acc[NTL][CT];
    const int64_t ho = ((int64_t)bh * P + p0 + tile_col<CT>(l16, 0)) * N + 8 * q;
    auto hn = [&](int t, int ct) { return ho + ct * 4 * N + (t >> 1) * 32 + (t & 1) * 4; };
#pragma unroll
    for (int t = 0; t < NTL; ++t)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
            acc[t][ct] = a.h0 ? ld4(a.h0 + hn(t, ct))
                              : f32x4{0.f, 0.f, 0.f, 0.f};

    const int rsk = G * N * 2, rsx = H * P * 2;
    auto rows_left = [&](int c) { return (int)min((int64_t)L, Tn - (int64_t)c * L); };
    auto key_rsrc = [&](const void* base, int c) {
        return make_rsrc(static_cast<const bf16*>(base) + ((tok0 + (int64_t)c * L) * G + g) * N,
                         (uint32_t)((rows_left(c) - 1) * rsk + N * 2));
    };
    auto x_rsrc = [&](const void* base, int c) {
        return make_rsrc(static_cast<const bf16*>(base) + ((tok0 + (int64_t)c * L) * H + h) * P,
                         (uint32_t)((rows_left(c) - 1) * rsx + P * 2));
    };
    auto item = [&](int c) { return (int64_t)(kb0 + c) * H + h; };
    auto fetch_k = [&](int c, bf16* kd) { dma_tile<N>(key_rsrc(a.B, c), kd, rsk, w, nw, lane); };
    auto fetch_q = [&](int c) { dma_tile<N>(key_rsrc(a.C, c), Qs, rsk, w, nw, lane); };
    auto fetch_tab = [&](int c) {
        const bf16* src = reinterpret_cast<const bf16*>(a.tab) + item(c) * (kFragTab + kFragVec);
        dma_run(make_rsrc(src, kFragTab * 2), reinterpret_cast<char*>(Sf), kFragTab / 512, w, nw, lane);
        if (w == 0 && lane < 32)
            dma_run(make_rsrc(src + kFragTab, 2 * L * 4), reinterpret_cast<char*>(Vs), 1, 0, 1, lane);
    };
    const int xo = rows_off<CT>(lane, rsx, p0);
    const unsigned sel = quad_sel(lane);
    const bool upper = (lane & 2) != 0;
    u32x2v xr[4][CT];  // x of the chunk, as loaded
    auto fetch_x = [&](int c) {
        const brsrc r = x_rsrc(a.x, c);
#pragma unroll
        for (int it = 0; it < 4; ++it) load_tile<CT>(r, xr[it], xo, it, rsx);
    };

    // lane offsets (elements) of the fragment reads; further fragments differ by an exchange of
    // piece bits and by whole row tiles
    const int ka = l16 * N + ((q ^ (l16 & SWZ)) << 3);
    const int tr = 4 * q + (l16 >> 2);
    const int kt = tr * N + (((l16 & 3) ^ (tr & SWZ)) << 3);
    // rows n of tile t (see acc), tokens as the accumulators hold them
    auto frag_t = [&](const bf16* tile, int t) {
        const bf16* p = tile + (kt ^ ((t >> 1) << 5)) + 4 * (t & 1);
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(ds_tr16(p), ds_tr16(p + 16 * N), 0, 1, 2, 3, 4, 5, 6, 7));
    };

    if (nc > 0) {
        fetch_k(0, K0);
        fetch_q(0);
        fetch_tab(0);
        fetch_x(0);
    }
    auto chunk = [&](int c, const bf16* Ks, bf16* Kn) {
        wave_meet(true);  // the chunk's tiles have landed
        const bool more = c + 1 < nc;
        if (KB == 2 && more) fetch_k(c + 1, Kn);

        // K h^T in three terms, Q h^T in two (enough for a bfloat16 y)
        f32x4 v[4][CT], yq[4][CT];
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) v[it][ct] = yq[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            Sp<bf16> hs[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) split8(join(acc[2 * ks][ct], acc[2 * ks + 1][ct]), hs[ct]);
            bf16x8 kf[4], qf[4];
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                kf[it] = ld8(Ks + (ka ^ (ks << 5)) + it * 16 * N);
                qf[it] = ld8(Qs + (ka ^ (ks << 5)) + it * 16 * N);
            }
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int it = 0; it < 4; ++it)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        v[it][ct] = mma(v[it][ct], kf[it], hs[ct].t[k]);
                        if (k < 2) yq[it][ct] = mma(yq[it][ct], qf[it], hs[ct].t[k]);
                    }
        }
        wave_meet(false);  // every wave is done with Q
        if (more) fetch_q(c + 1);

        // R, then r = R - S beta R
        Sp<bf16> b2[2][CT];
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const f32x4 ec = ld4(Vs + it * 16 + 4 * q);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                v[it][ct] = floats(quad_t(xr[it][ct], sel, upper)) - ec * v[it][ct];
                yq[it][ct] *= ec;
            }
        }
        if (more) fetch_x(c + 1);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) split8(join(v[2 * t][ct], v[2 * t + 1][ct]), b2[t][ct]);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 3; ++k) {  // term of S
                bf16x8 sf[4];
#pragma unroll
                for (int it = 2 * t; it < 4; ++it) sf[it] = frag_tab5(Sf + k * 5 * 512, it, t, lane);
#pragma unroll
                for (int m = 0; m < 3 - k; ++m)
#pragma unroll
                    for (int it = 2 * t; it < 4; ++it)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) v[it][ct] = mma(v[it][ct], sf[it], b2[t][ct].t[m]);
            }
        // Y = e^c Q h^T + M beta r
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) split8<2>(join(v[2 * t][ct], v[2 * t + 1][ct]), b2[t][ct]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // term of M
                bf16x8 mf[4];
#pragma unroll
                for (int it = 2 * t; it < 4; ++it) mf[it] = frag_tab5(Mf + k * 5 * 512, it, t, lane);
#pragma unroll
                for (int m = 0; m < 2 - k; ++m)
#pragma unroll
                    for (int it = 2 * t; it < 4; ++it)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) yq[it][ct] = mma(yq[it][ct], mf[it], b2[t][ct].t[m]);
            }
        }
        // e^{c_L - c} u as operands
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const f32x4 sa = ld4(Vs + L + 32 * t + 4 * q), sb = ld4(Vs + L + 32 * t + 16 + 4 * q);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) split8(join(v[2 * t][ct] * sa, v[2 * t + 1][ct] * sb), b2[t][ct]);
        }
        const float el = Vs[L - 1];
        wave_meet(false);  // every wave is done with the tables
        if (more) fetch_tab(c + 1);
        {
            const brsrc ry = x_rsrc(a.y, c);
#pragma unroll
            for (int it = 0; it < 4; ++it) store_tile<CT>(ry, yq[it], xo, it, rsx, sel, upper);
        }
        // h' = e^{c_L} h + K^T (e^{c_L - c} u), four row tiles side by side: a product on an
        // accumulator waits for the one before it
#pragma unroll
        for (int t4 = 0; t4 < NTL; t4 += 4) {
            bf16x8 kf[4][2];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) kf[t][ks] = frag_t(Ks + ks * 32 * N, t4 + t);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) acc[t4 + t][ct] *= el;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int k = 0; k < 3; ++k)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct)
                            acc[t4 + t][ct] = mma(acc[t4 + t][ct], kf[t][ks], b2[ks][ct].t[k]);
        }
        if (KB == 1 && more) {
            wave_meet(false);  // every wave is done with K
            fetch_k(c + 1, K0);
        }
    };
    if (KB == 2) {
        for (int c = 0; c < nc; c += 2) {
            chunk(c, K0, K1);
            if (c + 1 < nc) chunk(c + 1, K1, K0);
        }
    } else {
        for (int c = 0; c < nc; ++c) chunk(c, K0, K0);
    }
    if (a.hT) {
#pragma unroll
        for (int t = 0; t < NTL; ++t)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
                st4(a.hT + hn(t, ct), acc[t][ct]);
    }
}

// ---------------------------------------------------------------------------
// k_delta_team: the same walk by a team of 8 waves per 16 CT columns, for few chains and for the
// backward's first walk (SAVE).  Four waves own a quarter of the state each and carry what the
// next chunk waits for: K h^T in partial sums (their own state is the operand, straight from the
// accumulators), R, r and the state's update.  The other four, one beside each on its SIMD, do
// the rest meanwhile: every transfer into LDS, Q h^T, Y and its store.  Four exchanges per chunk.
// Bound by a chunk's latency: one row of 65536 tokens, 32 heads of 64, dstate 256 (128 teams), 2.4 ms,
// 2.3 us a chunk; without its transfers 1.9.  LDS moves 390 KB a chunk, 1.3 us at 128 bytes a
// cycle.  (Four waves doing all of it in turn: 2.8 ms.  Keys and tables straight to the
// registers of the one wave that reads them: 3.1 ms, their scattered rows choke the
// address unit.  Lines touched two chunks ahead: 2.7 ms, of the same cause.)
// SAVE = true writes the residuals r, the state entering every chunk, e^c K h^T and the per-token
// e^c dY . h Q (all terms) instead of y and hT; it reads no M.
// ---------------------------------------------------------------------------
// what the two team walks share: the chunk addresses of one (row, head) and the lane's offsets
template <int N, int CT>
struct Team {
    static constexpr int OT = N / 64;  // state tiles per wave: OT w .. OT w + OT - 1
    int lane, w, l16, q, H, G, P, h, row, g, nc, kb0, sl, bh, p0, rsk, rsx, xo;  // w: wave of four
    int64_t Tn, tok0, ho;
    unsigned sel;
    bool upper;
    int ka, kt;
    const Args& a;
    __device__ __forceinline__ Team(const Args& a_) : a(a_) {
        constexpr int SWZ = Dma<N>::SWZ;
        lane = threadIdx.x & 63; w = wave_id() & 3; l16 = lane & 15; q = lane >> 4;
        H = a.H; G = a.G; P = a.P;
        const int nsl = P / (16 * CT);
        const Item it = xcd_item(blockIdx.x, H, nsl, a.order);
        sl = it.sl; bh = it.bh;
        h = bh % H; row = bh / H; g = h / (H / G);
        Tn = a.rows.len(row); tok0 = a.rows.tok0(row); nc = a.rows.nchunks(row); kb0 = a.rows.kbase(row);
        p0 = sl * 16 * CT;
        rsk = G * N * 2; rsx = H * P * 2;
        xo = rows_off<CT>(lane, rsx, p0);
        sel = quad_sel(lane); upper = (lane & 2) != 0;
        ho = ((int64_t)bh * P + p0 + tile_col<CT>(l16, 0)) * N + 8 * q;
        ka = l16 * N + ((q ^ (l16 & SWZ)) << 3);
        const int tr = 4 * q + (l16 >> 2);
        kt = tr * N + (((l16 & 3) ^ (tr & SWZ)) << 3);
    }
    __device__ __forceinline__ int64_t hn(int t, int ct) const { return ho + ct * 4 * N + (t >> 1) * 32 + (t & 1) * 4; }
    __device__ __forceinline__ int rows_left(int c) const { return (int)min((int64_t)L, Tn - (int64_t)c * L); }
    __device__ __forceinline__ int64_t item(int c) const { return (int64_t)(kb0 + c) * H + h; }
    __device__ __forceinline__ brsrc key_rsrc(const void* base, int c) const {
        return make_rsrc(static_cast<const bf16*>(base) + ((tok0 + (int64_t)c * L) * G + g) * N,
                         (uint32_t)((rows_left(c) - 1) * rsk + N * 2));
    }
    __device__ __forceinline__ brsrc x_rsrc(const void* base, int c) const {
        return make_rsrc(static_cast<const bf16*>(base) + ((tok0 + (int64_t)c * L) * H + h) * P,
                         (uint32_t)((rows_left(c) - 1) * rsx + P * 2));
    }
    __device__ __forceinline__ void fetch_tile(const void* base, int c, bf16* dst) const {
        constexpr int RPI = 512 / N, PC = Dma<N>::PIECES;
        const brsrc r = key_rsrc(base, c);
#pragma unroll
        for (int k = 0; k < L / RPI / 4; ++k) {
            const int m = w + 4 * k, rw = m * RPI + lane / PC, j = (lane % PC) ^ (rw & Dma<N>::SWZ);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(dst + m * 512), 16, rw * rsk + j * 16, 0, 0, 0);
        }
    }
    // One transfer of no consequence (dst is written before it is read).  The compiler waits for
    // every transfer in flight before it reads an LDS array that none ever goes to; an array
    // that one goes to is waited for on its own account only.
    __device__ __forceinline__ void mark(bf16* dst) const {
        if (w == 0) dma_run(make_rsrc(a.tab, 1024), reinterpret_cast<char*>(dst), 1, 0, 1, lane);
    }
    // RUNS KiB of a chunk's tables and factors, which are ALL KiB, from the FROM-th on
    template <int ALL, int FROM, int RUNS>
    __device__ __forceinline__ void fetch_tab(int c, bf16* dst) const {
        const brsrc r = make_rsrc(reinterpret_cast<const bf16*>(a.tab) + (item(c) * ALL + FROM) * 512, RUNS * 1024);
#pragma unroll
        for (int k = 0; k < RUNS; k += 4)
            if (k + w < RUNS)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(dst + (k + w) * 512), 16, (k + w) * 1024 + lane * 16, 0,
                                                         0, 0);
    }
    // a chunk's 64 x 16 CT tile of x or dy: dst[token][16 CT]
    __device__ __forceinline__ void fetch_x(const void* base, int c, bf16* dst) const {
        const brsrc r = x_rsrc(base, c);
        if (w < 2 * CT)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(dst + w * 512), 16,
                                                     (w * 32 / CT + lane / (2 * CT)) * rsx + (p0 + 8 * (lane % (2 * CT))) * 2,
                                                     0, 0, 0);
    }
    // token tile `it` of it, in accumulator order (4 tokens of one column)
    __device__ __forceinline__ s16x4 x_tile(const bf16* src, int it, int ct) const {
        return ds_tr16(src + (it * 16 + 4 * q + (l16 >> 2)) * 16 * CT + 4 * CT * (l16 & 3) + 4 * ct);
    }
    // token tile w of a [token][H P] tensor
    __device__ __forceinline__ void store_rows(void* base, int c, const f32x4 (&v)[CT]) const {
        store_tile<CT>(x_rsrc(base, c), v, xo, w, rsx, sel, upper);
    }
    // the same in three terms
    __device__ __forceinline__ void store_rows3(void* hi, void* lo, void* ll, int c, const f32x4 (&v)[CT]) const {
        f32x4 r1[CT], r2[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            r1[ct] = rest16(v[ct]);
            r2[ct] = rest16(r1[ct]);
        }
        store_rows(hi, c, v);
        store_rows(lo, c, r1);
        store_rows(ll, c, r2);
    }
    // fragments: token tile `it`, key columns 32 ks on; state tile t, 32 tokens from tile row `p`
    __device__ __forceinline__ bf16x8 frag_rows16(const bf16* tile, int it, int ks) const {
        return ld8(tile + (ka ^ (ks << 5)) + it * 16 * N);
    }
    __device__ __forceinline__ bf16x8 frag_t(const bf16* tile, int t) const {
        const bf16* p = tile + (kt ^ ((t >> 1) << 5)) + 4 * (t & 1);
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(ds_tr16(p), ds_tr16(p + 16 * N), 0, 1, 2, 3, 4, 5, 6, 7));
    }
    // this wave's state tiles as operands, in pairs of tiles (dstate 64: one tile and zeros)
    static constexpr int OP = (OT + 1) / 2;
    __device__ __forceinline__ void split(const f32x4 (&acc)[OT][CT], Sp<bf16> (&sp)[OP][CT]) const {
        const f32x4 z = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int o = 0; o < OP; ++o)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                if (OT > 1) split8(join(acc[2 * o][ct], acc[2 * o + 1 < OT ? 2 * o + 1 : 0][ct]), sp[o][ct]);
                else split8(w & 1 ? join(z, acc[0][ct]) : join(acc[0][ct], z), sp[o][ct]);
            }
    }
    __device__ __forceinline__ int ks_of(int o) const { return OT > 1 ? OT / 2 * w + o : w >> 1; }
    // the first TS terms to LDS: dst[ks][term][ct][lane][8]
    template <int TS>
    __device__ __forceinline__ void put_state(bf16* dst, const Sp<bf16> (&sp)[OP][CT]) const {
#pragma unroll
        for (int o = 0; o < OP; ++o)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int k = 0; k < TS; ++k) {
                    bf16* d = dst + ((ks_of(o) * TS + k) * CT + ct) * 512 + lane * 8;
                    const bf16x8 v = sp[o][ct].t[k];
                    if (OT > 1) st8(d, v);
                    else st4(d + 4 * (w & 1), w & 1 ? __builtin_shufflevector(v, v, 4, 5, 6, 7)
                                                    : __builtin_shufflevector(v, v, 0, 1, 2, 3));
                }
    }
    // the product of a key tile with the state, this wave's part of its sum for all 4 token
    // tiles, to dst[wave][tile][ct][lane]; `sum` adds tile w up over the waves
    __device__ __forceinline__ void part_sums(const bf16* tile, const Sp<bf16> (&sp)[OP][CT], float* dst) const {
        f32x4 pv[4][CT];
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) pv[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
        bf16x8 kf[OP][4];
#pragma unroll
        for (int o = 0; o < OP; ++o)
#pragma unroll
            for (int it = 0; it < 4; ++it) kf[o][it] = frag_rows16(tile, it, ks_of(o));
#pragma unroll
        for (int o = 0; o < OP; ++o)
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int it = 0; it < 4; ++it)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) pv[it][ct] = mma(pv[it][ct], kf[o][it], sp[o][ct].t[k]);
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) st4(dst + ((w * 4 + it) * CT + ct) * 256 + lane * 4, pv[it][ct]);
    }
    __device__ __forceinline__ f32x4 sum(const float* src, int ct) const {
        f32x4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = ld4(src + ((k * 4 + w) * CT + ct) * 256 + lane * 4);
        return (v[0] + v[1]) + (v[2] + v[3]);
    }
    // token tile w's values to LDS operands dst[t][term][ct][lane][8] of TS terms
    template <int TS>
    __device__ __forceinline__ void put_rows(bf16* dst, const f32x4 (&v)[CT]) const {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            bf16x4 o[TS];
            split4<TS>(v[ct], o);
#pragma unroll
            for (int k = 0; k < TS; ++k) st4(dst + (((w >> 1) * TS + k) * CT + ct) * 512 + lane * 8 + 4 * (w & 1), o[k]);
        }
    }
    template <int TS>
    __device__ __forceinline__ bf16x8 get(const bf16* src, int t, int k, int ct) const {
        return ld8(src + ((t * TS + k) * CT + ct) * 512 + lane * 8);
    }
    // tile row w of a table of TERMS terms, columns 32 t on (t <= w / 2)
    template <int TERMS>
    __device__ __forceinline__ void table_row(const bf16* tab, bf16x8 (&f)[2][TERMS]) const {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (t > (w >> 1)) break;
            const int lo = w == 2 && t == 1 ? 4 : w == 0 ? 0 : (w < 3 ? w : 3 + t) * 512;
            const int hi = w < 3 && t == (w >> 1) && !(w & 1) ? lo : lo + 4;  // (no such block: zero)
#pragma unroll
            for (int k = 0; k < TERMS; ++k) {
                const bf16* tk = tab + k * 5 * 512 + lane * 8;
                u32x2 h2 = __builtin_bit_cast(u32x2, ld4(tk + hi));
                if (hi == lo) h2 = u32x2{0, 0};
                f[t][k] = join(ld4(tk + lo), __builtin_bit_cast(bf16x4, h2));
            }
        }
    }
    // o += that row times token operands src in LDS (ST terms), products of order below ST
    template <int TERMS, int ST>
    __device__ __forceinline__ void times_rows(f32x4 (&o)[CT], const bf16x8 (&f)[2][TERMS], const bf16* src) const {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (t > (w >> 1)) break;
            f32x4 p[CT];  // the second half of the products, beside the first
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) p[ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < TERMS; ++k)
#pragma unroll
                for (int m = 0; m < ST - k; ++m)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        f32x4& v = (k + m) & 1 ? p[ct] : o[ct];
                        v = mma(v, f[t][k], get<ST>(src, t, m, ct));
                    }
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) o[ct] += p[ct];
        }
    }
};
__device__ __forceinline__ f32x4 floats(s16x4 v) { return floats(__builtin_bit_cast(u32x2v, v)); }

template <int N, int CT, int KB, bool SAVE>
__global__ __launch_bounds__(512) void k_delta_team(Args a) {
    typedef Team<N, CT> TM;
    constexpr int KS = N / 32, TILE = Dma<N>::TILE, OT = TM::OT, OP = TM::OP;
    constexpr int QT = SAVE ? 3 : 2, MT = 2, UT = 2;  // terms of h, M and u in Y
    constexpr int ALL = (SAVE ? kFragTab2 : kFragTab) / 512 + 1, RUNS = SAVE ? 16 : ALL;  // (SAVE: S and the factors)
    __shared__ __attribute__((aligned(16))) bf16 K0[TILE];
    __shared__ __attribute__((aligned(16))) bf16 K1[KB == 2 ? TILE : 8];
    __shared__ __attribute__((aligned(16))) bf16 Qs[TILE];
    __shared__ __attribute__((aligned(16))) bf16 Sf[RUNS * 512];
    __shared__ __attribute__((aligned(16))) bf16 Ys[SAVE ? CT * 1024 : 8];
    // passed between the waves: partial sums, then (once they are read) the weighted u and u;
    // the state's operands for Q h^T; R
    constexpr int PF = 16 * CT * 512, HF = KS * QT * CT * 512, RF = 2 * 3 * CT * 512;
    __shared__ __attribute__((aligned(16))) bf16 Ex[PF + HF + RF];
    bf16 *Wf = Ex, *Uf = Wf + RF, *Hf = Ex + PF, *Rf = Hf + HF;
    float* Pf = reinterpret_cast<float*>(Ex);
    const bf16* Mf = Sf + 15 * 512;
    const float* Vs = reinterpret_cast<const float*>(Sf + (RUNS - 1) * 512);
    const TM tm(a);
    const int lane = tm.lane, w = tm.w, l16 = tm.l16, q = tm.q, nc = tm.nc, t0w = OT * w;
    if (nc > 0 && wave_id() >= 4) {
        auto bring = [&](int c) {
            tm.template fetch_tab<ALL, 0, SAVE ? 15 : ALL>(c, Sf);
            if (SAVE) {
                tm.template fetch_tab<ALL, ALL - 1, 1>(c, Sf + 15 * 512);
                tm.fetch_x(a.dy, c, Ys);
            }
        };
        tm.fetch_tile(a.B, 0, K0);
        tm.fetch_tile(a.C, 0, Qs);
        bring(0);
        tm.mark(Rf);
        f32x4 yq[CT], d;
        // what a chunk leaves to memory, sent on its way at the start of the next
        auto leave = [&](int c) {
            if (SAVE) {
                f32x4 e;
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = row_sum16(d[i]);
                const int t = w * 16 + 4 * q + (l16 & 3);
                const float dt = l16 & 2 ? (l16 & 1 ? e[3] : e[2]) : (l16 & 1 ? e[1] : e[0]);
                if (l16 < 4 && t < tm.rows_left(c))
                    a.fq[((int64_t)tm.sl * a.rows.nrows * a.H + tm.bh) * a.T + (int64_t)c * L + t] = dt;
            } else {
                tm.store_rows(a.y, c, yq);
            }
        };
        auto chunk = [&](int c, bf16* Kn) {
            const bool more = c + 1 < nc;
            wave_meet(true);  // the chunk's tiles have landed, the state's operands are in place
            if (c > 0) leave(c - 1);
            if (KB == 2 && more) tm.fetch_tile(a.B, c + 1, Kn);
            const f32x4 ec = ld4(Vs + w * 16 + 4 * q);
            // Q h^T of token tile w, two accumulators
            f32x4 y2[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) yq[ct] = y2[ct] = f32x4{0.f, 0.f, 0.f, 0.f};
            auto qh = [&](int from, int to) {
#pragma unroll
                for (int ks = from; ks < to; ++ks) {
                    const bf16x8 qf = tm.frag_rows16(Qs, w, ks);
#pragma unroll
                    for (int k = 0; k < QT; ++k)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) {
                            f32x4& yy = ks & 1 ? y2[ct] : yq[ct];
                            yy = mma(yy, qf, tm.template get<QT>(Hf, ks, k, ct));
                        }
                }
            };
            bf16x8 mf[2][MT];
            if (!SAVE) tm.template table_row<MT>(Mf, mf);
            f32x4 dy[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
                if (SAVE) dy[ct] = floats(tm.x_tile(Ys, w, ct));
            qh(0, KS - KS / 4);
            wave_meet(false);  // the partial sums are in place, the tables and dY in registers
            if (more) bring(c + 1);
            qh(KS - KS / 4, KS);
            wave_meet(false);  // R is in place, K^T in registers, Q is free
            if (more) {
                tm.fetch_tile(a.C, c + 1, Qs);
                if (KB == 1) tm.fetch_tile(a.B, c + 1, Kn);
            }
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) yq[ct] = ec * (yq[ct] + y2[ct]);
            d = f32x4{0.f, 0.f, 0.f, 0.f};
            if (SAVE) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) d += dy[ct] * yq[ct];
            }
            wave_meet(false);  // u is in place
            // Y = e^c Q h^T + M beta r
            if (!SAVE) tm.template times_rows<MT, UT>(yq, mf, Uf);
        };
        for (int c = 0; c < nc; c += 2) {
            chunk(c, KB == 2 ? K1 : K0);
            if (c + 1 < nc) chunk(c + 1, K0);
        }
        leave(nc - 1);
    } else if (wave_id() < 4) {
        f32x4 acc[OT][CT];
#pragma unroll
        for (int o = 0; o < OT; ++o)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
                acc[o][ct] = a.h0 ? ld4(a.h0 + tm.hn(t0w + o, ct)) : f32x4{0.f, 0.f, 0.f, 0.f};
        Sp<bf16> sp[OP][CT];
        tm.split(acc, sp);
        if (nc > 0) tm.template put_state<QT>(Hf, sp);
        u32x2v xr[CT];  // x of the chunk's token tile w, as loaded
        if (nc > 0) load_tile<CT>(tm.x_rsrc(a.x, 0), xr, tm.xo, w, tm.rsx);
        auto chunk = [&](int c, const bf16* Ks) {
            wave_meet(false);  // the chunk's tiles have landed
            tm.part_sums(Ks, sp, Pf);
            if (SAVE) {
                const int64_t so = (tm.item(c) - tm.bh) * a.P * N;
#pragma unroll
                for (int o = 0; o < OT; o += 2)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        bf16x8 hi;
                        s16x8 lo;
                        split_state(join(acc[o][ct], acc[o + 1 < OT ? o + 1 : o][ct]), hi, lo);
                        bf16* hp = static_cast<bf16*>(a.hin) + so + tm.hn(t0w + o, ct);
                        short* lp = a.hlo + so + tm.hn(t0w + o, ct);
                        if (OT > 1) {
                            st8(hp, hi);
                            *reinterpret_cast<s16x8*>(lp) = lo;
                        } else {
                            st4(hp, __builtin_shufflevector(hi, hi, 0, 1, 2, 3));
                            *reinterpret_cast<s16x4*>(lp) = __builtin_shufflevector(lo, lo, 0, 1, 2, 3);
                        }
                    }
            }
            const f32x4 ec = ld4(Vs + w * 16 + 4 * q), ew0 = ld4(Vs + L + w * 16 + 4 * q);
            f32x4 bt = f32x4{1.f, 1.f, 1.f, 1.f};
            if (SAVE) bt = ld4(Vs + 2 * L + w * 16 + 4 * q);
            const float el = Vs[L - 1];
            f32x4 v[CT], rb[CT], uw[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) v[ct] = floats(quad_t(xr[ct], tm.sel, tm.upper));
            // (no branch: the loads in flight can then be counted)
            load_tile<CT>(tm.x_rsrc(a.x, min(c + 1, nc - 1)), xr, tm.xo, w, tm.rsx);
            bf16x8 sf[2][3];
            tm.template table_row<3>(Sf, sf);
            wave_meet(false);  // the partial sums are in place
            // R = X - e^c K h^T of token tile w
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const f32x4 kh = ec * tm.sum(Pf, ct);
                if (SAVE) st4(a.kh + kh_at<CT>(tm.item(c), a.P, tm.sl, w, ct, lane), kh);
                v[ct] -= kh;
                rb[ct] = v[ct] * bt;
            }
            tm.template put_rows<3>(Rf, rb);
            bf16x8 kf[2][OT];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int o = 0; o < OT; ++o) kf[ks][o] = tm.frag_t(Ks + ks * 32 * N, t0w + o);
            wave_meet(false);  // R is in place
            // r = R - S beta R, over the tiles up to w
            tm.template times_rows<3, 3>(v, sf, Rf);
            const f32x4 ew = ew0 * bt;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                rb[ct] = v[ct] * bt;
                uw[ct] = v[ct] * ew;
            }
            tm.template put_rows<3>(Wf, uw);
            if (!SAVE) tm.template put_rows<UT>(Uf, rb);
#pragma unroll
            for (int o = 0; o < OT; ++o)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) acc[o][ct] *= el;
            wave_meet(false);  // the weighted u is in place
            // h' = e^{c_L} h + K^T (e^{c_L - c} u) of this wave's tiles
            bf16x8 wf[2][3][CT];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int k = 0; k < 3; ++k)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) wf[ks][k][ct] = tm.template get<3>(Wf, ks, k, ct);
#pragma unroll
            for (int p = 0; p < OP; ++p)  // (a pair of tiles is split while the next is multiplied)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                    for (int k = 0; k < 3; ++k)
#pragma unroll
                        for (int o = 2 * p; o < 2 * p + (OT > 1 ? 2 : 1); ++o)
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct) acc[o][ct] = mma(acc[o][ct], kf[ks][o], wf[ks][k][ct]);
            tm.split(acc, sp);
            if (c + 1 < nc) tm.template put_state<QT>(Hf, sp);
            if (SAVE) {
                tm.store_rows3(a.r, a.rlo, a.rll, c, v);
            }
        };
        for (int c = 0; c < nc; c += 2) {
            chunk(c, K0);
            if (c + 1 < nc) chunk(c + 1, KB == 2 ? K1 : K0);
        }
        if (!SAVE && a.hT) {
#pragma unroll
            for (int o = 0; o < OT; ++o)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) st4(a.hT + tm.hn(t0w + o, ct), acc[o][ct]);
        }
    }
}

// ---------------------------------------------------------------------------
// k_delta_adj: the adjoint walk by the same teams (chunks in reverse, dh^T in accumulators); the
// tables' transposes are read from the same fragments by transposing loads.  Outputs as
// k_delta_rev.  Four waves, which share every product.  Bound by a chunk's latency: 2 rows of 2048
// tokens, 48 heads of 64, dstate 128, in 188 us, 5.9 us a chunk (the first walk: 129 us).
// ---------------------------------------------------------------------------
template <int N, int CT, int KB>
__global__ __launch_bounds__(256) void k_delta_adj(Args a) {
    constexpr int KS = N / 32, TILE = Dma<N>::TILE, OT = Team<N, CT>::OT, TABN = kFragTab2 + kFragVec;
    __shared__ __attribute__((aligned(16))) bf16 K0[TILE];
    __shared__ __attribute__((aligned(16))) bf16 K1[KB == 2 ? TILE : 8];
    __shared__ __attribute__((aligned(16))) bf16 Qs[TILE];
    __shared__ __attribute__((aligned(16))) bf16 Sf[TABN];
    __shared__ __attribute__((aligned(16))) bf16 Ys[CT * 1024];
    constexpr int HF = KS * 3 * CT * 512, RF = 2 * 3 * CT * 512;
    __shared__ __attribute__((aligned(16))) bf16 Ex[HF + 3 * RF];  // operands passed between the waves
    const bf16* Mf = Sf + 3 * 5 * 512;
    const float* Vs = reinterpret_cast<const float*>(Sf + TABN - kFragVec);
    bf16 *Hf = Ex, *Rf = Hf + HF, *Wf = Rf + RF, *Yf = Wf + RF;  // Wf: -e^c dX, Yf: e^c dY
    const Team<N, CT> tm(a);
    const int lane = tm.lane, w = tm.w, l16 = tm.l16, q = tm.q, nc = tm.nc, t0w = OT * w;
    const int64_t BH = (int64_t)a.rows.nrows * a.H;

    f32x4 acc[OT][CT];
#pragma unroll
    for (int o = 0; o < OT; ++o)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
            acc[o][ct] = a.dhT ? ld4(a.dhT + tm.hn(t0w + o, ct)) : f32x4{0.f, 0.f, 0.f, 0.f};
    const int ft = (4 * q + (l16 >> 2) + 16 * (l16 & 3)) * 8;  // four columns of a block's row, in a fragment
    // rows of tile w of the table's transpose, columns 32 t on (t >= w / 2)
    auto frag_up = [&](const bf16* tab, int t) {
        const s16x4 z = s16x4{0, 0, 0, 0};
        auto at = [&](int i) { return i == 2 && w == 2 ? 4 : i == 0 ? 0 : (i < 3 ? i : 3 + (w >> 1)) * 512 + 4 * (w & 1); };
        const s16x4 lo = 2 * t >= w ? ds_tr16(tab + at(2 * t) + ft) : z;
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, ds_tr16(tab + at(2 * t + 1) + ft), 0, 1, 2, 3, 4,
                                                                  5, 6, 7));
    };
    // dh' of a chunk, in accumulators: stored for the gradients of B
    constexpr int OP = (OT + 1) / 2;
    auto leave = [&](int c) {
        const int64_t lo = (tm.item(c) - tm.bh) * a.P * N;
#pragma unroll
        for (int o = 0; o < OP; ++o)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                Sp<bf16> ov;
                split8<1>(join(acc[2 * o][ct], acc[2 * o + 1 < OT ? 2 * o + 1 : 2 * o][ct]), ov);
                bf16* lp = static_cast<bf16*>(a.lin) + lo + tm.hn(t0w + 2 * o, ct);
                if (OT > 1) st8(lp, ov.t[0]);
                else st4(lp, __builtin_shufflevector(ov.t[0], ov.t[0], 0, 1, 2, 3));
            }
    };
    if (nc > 0) {
        tm.fetch_tile(a.B, nc - 1, K0);
        tm.template fetch_tab<TABN / 512, 0, TABN / 512>(nc - 1, Sf);
        tm.fetch_x(a.dy, nc - 1, Ys);
        tm.mark(Rf);
        Sp<bf16> sp[OP][CT];
        tm.split(acc, sp);
        tm.template put_state<3>(Hf, sp);
        leave(nc - 1);
    }
    auto chunk = [&](int c, const bf16* Ks, bf16* Kn) {
        const bool more = c > 0;
        wave_meet(true);  // the chunk's tiles have landed, the adjoint's operands are in place
        tm.fetch_tile(a.C, c, Qs);  // read last in the chunk
        if (KB == 2 && more) tm.fetch_tile(a.B, c - 1, Kn);
        // the state entering this chunk, e^c K h^T and r of token tile w, for the decays' gradients: consumed
        // at the end
        bf16x8 hi[OP][CT];
        s16x8 hl[OP][CT];
        {
            const int64_t so = (tm.item(c) - tm.bh) * a.P * N;
#pragma unroll
            for (int o = 0; o < OP; ++o)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const bf16* hp = static_cast<const bf16*>(a.hin) + so + tm.hn(t0w + 2 * o, ct);
                    const short* lp = a.hlo + so + tm.hn(t0w + 2 * o, ct);
                    if (OT > 1) {
                        hi[o][ct] = ld8(hp);
                        hl[o][ct] = *reinterpret_cast<const s16x8*>(lp);
                    } else {
                        hi[o][ct] = join(ld4(hp), ld4(hp));
                        const s16x4 l4 = *reinterpret_cast<const s16x4*>(lp);
                        hl[o][ct] = __builtin_shufflevector(l4, l4, 0, 1, 2, 3, 4, 5, 6, 7);
                    }
                }
        }
        f32x4 kh[CT];
        u32x2v rt[3][CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) kh[ct] = ld4(a.kh + kh_at<CT>(tm.item(c), a.P, tm.sl, w, ct, lane));
        load_tile<CT>(tm.x_rsrc(a.r, c), rt[0], tm.xo, w, tm.rsx);
        load_tile<CT>(tm.x_rsrc(a.rlo, c), rt[1], tm.xo, w, tm.rsx);
        load_tile<CT>(tm.x_rsrc(a.rll, c), rt[2], tm.xo, w, tm.rsx);
        // dU = e^{c_L - c} K dh'^T + M^T dY of token tile w
        f32x4 v[CT], v2[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) v[ct] = v2[ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const bf16x8 kf = tm.frag_rows16(Ks, w, ks);
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    f32x4& vv = ks & 1 ? v2[ct] : v[ct];
                    vv = mma(vv, kf, tm.template get<3>(Hf, ks, k, ct));
                }
        }
        const f32x4 ec = ld4(Vs + w * 16 + 4 * q), ew = ld4(Vs + L + w * 16 + 4 * q),
                    bt = ld4(Vs + 2 * L + w * 16 + 4 * q);
        f32x4 rb[CT], yw[CT], kd[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            kd[ct] = v[ct] = ew * (v[ct] + v2[ct]);
            yw[ct] = ec * floats(tm.x_tile(Ys, w, ct));
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (t < (w >> 1)) continue;
                const bf16x8 dyf = __builtin_bit_cast(
                    bf16x8, __builtin_shufflevector(tm.x_tile(Ys, 2 * t, ct), tm.x_tile(Ys, 2 * t + 1, ct), 0, 1, 2, 3, 4,
                                                    5, 6, 7));
#pragma unroll
                for (int k = 0; k < 3; ++k) v[ct] = mma(v[ct], frag_up(Mf + k * 5 * 512, t), dyf);
            }
            rb[ct] = v[ct] * bt;
        }
        tm.template put_rows<3>(Rf, rb);
        tm.template put_rows<3>(Yf, yw);
        wave_meet(false);  // beta dU is in place; every wave is done with dY
        if (more) tm.fetch_x(a.dy, c - 1, Ys);
        // z = dU - S^T (beta dU), over the tiles from w on
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (t < (w >> 1)) continue;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const bf16x8 f = frag_up(Sf + k * 5 * 512, t);
#pragma unroll
                for (int m = 0; m < 3 - k; ++m)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) v[ct] = mma(v[ct], f, tm.template get<3>(Rf, t, m, ct));
            }
        }
        f32x4 dx[CT], wv[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            dx[ct] = v[ct] * bt;
            wv[ct] = dx[ct] * -ec;
        }
        tm.template put_rows<3>(Wf, wv);
        const float el = Vs[L - 1];
        wave_meet(true);  // dX is in place, Q has landed; every wave is done with the tables
        if (more) {
            tm.template fetch_tab<TABN / 512, 0, TABN / 512>(c - 1, Sf);
        }
        tm.store_rows3(a.z, a.zlo, a.zll, c, v);
        tm.store_rows(a.dx, c, dx);
        {  // of the decays' gradients: e^c dX . h K and u . e^{c_L - c} dh' K of the tile's tokens
            f32x4 f = f32x4{0.f, 0.f, 0.f, 0.f}, g = f;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                f32x4 r = floats(quad_t(rt[2][ct], tm.sel, tm.upper));
                r += floats(quad_t(rt[1][ct], tm.sel, tm.upper));
                r += floats(quad_t(rt[0][ct], tm.sel, tm.upper));
                f += kh[ct] * dx[ct];
                g += r * bt * kd[ct];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i] = row_sum16(f[i]);
                g[i] = row_sum16(g[i]);
            }
            const int t = w * 16 + 4 * q + (l16 & 3);
            const bool o1 = l16 & 1, o2 = l16 & 2;
            const int64_t at = ((int64_t)tm.sl * BH + tm.bh) * a.T + (int64_t)c * L + t;
            if (l16 < 4 && t < tm.rows_left(c)) {
                a.fk[at] = o2 ? (o1 ? f[3] : f[2]) : (o1 ? f[1] : f[0]);
                a.dj[at] = o2 ? (o1 ? g[3] : g[2]) : (o1 ? g[1] : g[0]);
            }
            // and e^{c_L} <dh', h> over this wave's tiles
            float s = 0.f;
#pragma unroll
            for (int o = 0; o < OP; ++o)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const f32x8 av = join(acc[2 * o][ct], acc[2 * o + 1 < OT ? 2 * o + 1 : 2 * o][ct]);
#pragma unroll
                    for (int i = 0; i < (OT > 1 ? 8 : 4); ++i) s += join_state(hi[o][ct][i], hl[o][ct][i]) * av[i];
                }
            s = row_sum16(s);
            s += __shfl_xor(s, 16, 64);
            s += __shfl_xor(s, 32, 64);
            if (lane == 0) a.tot[(int64_t)(tm.sl * 4 + w) * a.ntab * a.H + tm.item(c)] = s * el;
        }
        // dh = e^{c_L} dh' - K^T (e^c dX) + Q^T (e^c dY) of this wave's tiles
#pragma unroll
        for (int o = 0; o < OT; ++o)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) acc[o][ct] *= el;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            bf16x8 kf[OT], qf[OT];
#pragma unroll
            for (int o = 0; o < OT; ++o) {
                kf[o] = tm.frag_t(Ks + ks * 32 * N, t0w + o);
                qf[o] = tm.frag_t(Qs + ks * 32 * N, t0w + o);
            }
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const bf16x8 wf = tm.template get<3>(Wf, ks, k, ct), yf = tm.template get<3>(Yf, ks, k, ct);
#pragma unroll
                    for (int o = 0; o < OT; ++o) acc[o][ct] = mma(acc[o][ct], kf[o], wf);
#pragma unroll
                    for (int o = 0; o < OT; ++o) acc[o][ct] = mma(acc[o][ct], qf[o], yf);
                }
        }
        if (more) {
            Sp<bf16> sp[OP][CT];
            tm.split(acc, sp);
            tm.template put_state<3>(Hf, sp);
            leave(c - 1);
        }
        if (KB == 1 && more) {
            wave_meet(false);  // every wave is done with K
            tm.fetch_tile(a.B, c - 1, Kn);
        }
    };
    for (int c = nc - 1; c >= 0; c -= 2) {
        chunk(c, K0, KB == 2 ? K1 : K0);
        if (c > 0) chunk(c - 1, KB == 2 ? K1 : K0, K0);
    }
    if (a.dh0) {
#pragma unroll
        for (int o = 0; o < OT; ++o)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) st4(a.dh0 + tm.hn(t0w + o, ct), acc[o][ct]);
    }
}

// ---------------------------------------------------------------------------
// k_delta_rev: the adjoint walk, chunks in reverse; the same slices and layout, the adjoint
// state dh^T[n][p] in accumulators.  Writes dx, z, dh' of every chunk (problem dtype), for the
// decays' gradients the per-token e^c dX . h K and D and e^{c_L} <dh', h> of every chunk, and dh0.
// ---------------------------------------------------------------------------
template <typename T, int N>
__global__ __launch_bounds__(256) void k_delta_rev(Args a, int waves) {
    typedef Cfg<T, N> CF;
    constexpr int CT = 1;
    constexpr int NP = CF::NP, LDK = CF::LDK, NTL = N / 16, KS = NP / 32, NT = CF::NT;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), l16 = lane & 15, q = lane >> 4;
    const int H = a.H, G = a.G, P = a.P;
    const int SW = 16 * CT * waves, ldx = CF::ldx(SW);
    T* Ks = reinterpret_cast<T*>(smem);
    T* Qs = CF::SHARE ? Ks : Ks + CF::KT;
    T* Sf = Qs + CF::KT;
    T* Mf = Sf + NT * kFrag * 512;
    T* Xs = Mf + NT * kFrag * 512;
    T* Ys = Xs + L * ldx;  // dY rows, then z
    float* ecs = reinterpret_cast<float*>(Ys + L * ldx);
    float* ews = ecs + L;
    float* bts = ews + L;
    float* dots = bts + L;       // [wave][token]
    float* dots2 = dots + 4 * L;

    const int nsl = P / SW, BH = a.rows.nrows * H;
    const int sl = (int)(blockIdx.x % (unsigned)nsl);
    const int64_t bh = blockIdx.x / (unsigned)nsl;
    const int h = (int)(bh % H), row = (int)(bh / H), g = h / (H / G);
    const int64_t Tn = a.rows.len(row), tok0 = a.rows.tok0(row);
    const int nc = a.rows.nchunks(row), kb0 = a.rows.kbase(row);
    const int p0 = sl * SW, pw = w * 16 * CT;
    const bool on = w < waves;  // the others stage only

    f32x4 acc[NTL][CT];  // dh^T
#pragma unroll
    for (int t = 0; t < NTL; ++t)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
            acc[t][ct] = a.dhT && on ? ld4(a.dhT + (bh * P + p0 + pw + ct * 16 + l16) * N + t * 16 + 4 * q)
                               : f32x4{0.f, 0.f, 0.f, 0.f};

    // the state entering a chunk, for <dh', h>: asked for with the chunk's inputs (dstate 256 leaves
    // no registers to wait in)
    constexpr bool AHEAD = N <= 128;
    typename V4<T>::type hi[NTL][CT];
    s16x4 lo[NTL][CT];
    auto load_h = [&](int c) {
        const int64_t ho = (((int64_t)(kb0 + c) * H + h) * P + p0 + pw) * N;
#pragma unroll
        for (int t = 0; t < NTL; ++t)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int64_t o = ho + (ct * 16 + l16) * N + t * 16 + 4 * q;
                hi[t][ct] = ld4(static_cast<const T*>(a.hin) + o);
                if (NT > 1) lo[t][ct] = *reinterpret_cast<const s16x4*>(a.hlo + o);
            }
    };
    Staged<T, N, CT, NT, true> in;
    if (nc > 0) {
        in.load(a, row, h, nc - 1, p0, SW, true);
        if (AHEAD && on) load_h(nc - 1);
    }
    for (int c = nc - 1; c >= 0; --c) {
        const int64_t t0 = tok0 + (int64_t)c * L;
        const int n = (int)min((int64_t)L, Tn - (int64_t)c * L);
        const int64_t e = (int64_t)(kb0 + c) * H + h;
        float s = 0.f;  // <dh', h> over this wave's columns
        if (on) {
            if (!AHEAD) load_h(c);
#pragma unroll
            for (int t = 0; t < NTL; ++t)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (std::is_same<T, bf16>::value) s += join_state(hi[t][ct][i], lo[t][ct][i]) * acc[t][ct][i];
                        else s += hi[t][ct][i] * acc[t][ct][i];
                    }
            s = row_sum16(s);
            s += __shfl_xor(s, 16, 64);
            s += __shfl_xor(s, 32, 64);
        }
        wave_meet(false);  // the previous chunk's tiles are no longer read
        in.put(Ks, Qs, Xs, Ys, Sf, Mf, ecs, SW, true);
        wave_meet(false);
        if (on && lane == 0) a.tot[(int64_t)(sl * waves + w) * a.ntab * H + e] = s * ecs[L - 1];
        if (c > 0) {
            in.load(a, row, h, c - 1, p0, SW, true);
            if (AHEAD && on) load_h(c - 1);
        }
        Sp<T> b2[2][CT];
        if (on) {
            T* lp = static_cast<T*>(a.lin) + (e * P + p0 + pw) * N;
#pragma unroll
            for (int t = 0; t < NTL; ++t)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    typename V4<T>::type o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = from_f<T>(acc[t][ct][i]);
                    st4(lp + (ct * 16 + l16) * N + t * 16 + 4 * q, o);
                }
        // dU = e^{c_L - c} K dh'^T + M^T dY
        f32x4 v[4][CT];
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) v[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            Sp<T> hs[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
                split8(join(acc[2 * ks][ct], 2 * ks + 1 < NTL ? acc[2 * ks + 1 < NTL ? 2 * ks + 1 : 0][ct]
                                                              : f32x4{0.f, 0.f, 0.f, 0.f}),
                       hs[ct]);
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const auto fr = frag_k(Ks, LDK, it * 16 + l16, ks * 32, q);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) v[it][ct] = mma_es<3>(v[it][ct], fr, hs[ct]);
            }
        }
        typename V8<T>::type dyf[2][CT];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
                dyf[t][ct] = frag_rows_split(Ys, ldx, 32 * t + 4 * q, 32 * t + 16 + 4 * q, pw + ct * 16, lane);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = it * 16 + 4 * q + i;
                float dot = 0.f;  // D = u . e^{c_L - c} dh' K
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    v[it][ct][i] *= ews[t];
                    float r = to_f(Xs[t * ldx + pw + ct * 16 + l16]);
                    if (NT > 1 && t < n) {
                        const int64_t o = ((t0 + t) * H + h) * P + p0 + pw + ct * 16 + l16;
                        r += to_f(static_cast<const T*>(a.rlo)[o]) + to_f(static_cast<const T*>(a.rll)[o]);
                    }
                    dot += r * bts[t] * v[it][ct][i];
                }
                dot = row_sum16(dot);
                if (l16 == 0) dots2[w * L + t] = dot;
            }
#pragma unroll
            for (int t = it / 2; t < 2; ++t) {
                const Sp<T> mf = frag_tab<T, NT>(Mf, frag_up(it, t), lane);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int k2 = 0; k2 < NT; ++k2) v[it][ct] = mma(v[it][ct], mf.t[k2], dyf[t][ct]);
            }
        }
        // z = dU - S^T (beta dU)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                f32x4 lo = v[2 * t][ct], hi = v[2 * t + 1][ct];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lo[i] *= bts[32 * t + 4 * q + i];
                    hi[i] *= bts[32 * t + 16 + 4 * q + i];
                }
                split8(join(lo, hi), b2[t][ct]);
            }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            f32x4 d[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) d[ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = it / 2; t < 2; ++t) {
                const Sp<T> sf = frag_tab<T, NT>(Sf, frag_up(it, t), lane);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) d[ct] = mma_ss<3>(d[ct], sf, b2[t][ct]);
            }
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) v[it][ct] -= d[ct];
        }
        // dX = beta z, its dot with e^c h K; the tiles leave through LDS (own columns)
        f32x4 kh[4][CT];
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) kh[it][ct] = ld4(a.kh + kh_at<CT>(e, P, (p0 + pw) / (16 * CT), it, ct, lane));
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = it * 16 + 4 * q + i;
                float dot = 0.f;
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const int o = t * ldx + pw + ct * 16 + l16;
                    const float dxv = bts[t] * v[it][ct][i];
                    dot += dxv * kh[it][ct][i];
                    Xs[o] = from_f<T>(dxv);
                    Ys[o] = from_f<T>(v[it][ct][i]);
                    if (NT > 1 && t < n) {
                        const int64_t zo = ((t0 + t) * H + h) * P + p0 + pw + ct * 16 + l16;
                        const float rest = v[it][ct][i] - to_f(Ys[o]);
                        const T z1 = from_f<T>(rest);
                        static_cast<T*>(a.zlo)[zo] = z1;
                        static_cast<T*>(a.zll)[zo] = from_f<T>(rest - to_f(z1));
                    }
                    v[it][ct][i] = dxv;
                }
                dot = row_sum16(dot);
                if (l16 == 0) dots[w * L + t] = dot;
            }
        // dh = e^{c_L} dh' - K^T (e^c dX) + Q^T (e^c dY)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                f32x4 lo = v[2 * t][ct], hi = v[2 * t + 1][ct];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lo[i] *= -ecs[32 * t + 4 * q + i];
                    hi[i] *= -ecs[32 * t + 16 + 4 * q + i];
                }
                split8(join(lo, hi), b2[t][ct]);
            }
        const float el = ecs[L - 1];
#pragma unroll
        for (int t = 0; t < NTL; ++t) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) acc[t][ct] *= el;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const auto kf = frag_rows_split(Ks, LDK, ks * 32 + 4 * q, ks * 32 + 16 + 4 * q, t * 16, lane);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) acc[t][ct] = mma_es<3>(acc[t][ct], kf, b2[ks][ct]);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                f32x8 d;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] = to_f(dyf[t][ct][i]) * ecs[32 * t + 16 * (i >> 2) + 4 * q + (i & 3)];
                split8(d, b2[t][ct]);
            }
        }
        if (CF::SHARE) {
            wave_meet(false);
            stage_rows(static_cast<const T*>(a.C) + (t0 * G + g) * N, (int64_t)G * N, Qs, LDK, n, N, NP, tid, 256);
        }
        wave_meet(false);
        if (on) {
#pragma unroll
        for (int t = 0; t < NTL; ++t)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const auto qf = frag_rows_split(Qs, LDK, ks * 32 + 4 * q, ks * 32 + 16 + 4 * q, t * 16, lane);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) acc[t][ct] = mma_es<3>(acc[t][ct], qf, b2[ks][ct]);
            }
        }
        store_rows(static_cast<T*>(a.dx) + (t0 * H + h) * P + p0, (int64_t)H * P, Xs, ldx, n, SW, tid, 256);
        store_rows(static_cast<T*>(a.z) + (t0 * H + h) * P + p0, (int64_t)H * P, Ys, ldx, n, SW, tid, 256);
        for (int t = tid; t < n; t += 256) {
            float f = 0.f, g = 0.f;
            for (int k2 = 0; k2 < waves; ++k2) {
                f += dots[k2 * L + t];
                g += dots2[k2 * L + t];
            }
            const int64_t at = ((int64_t)sl * BH + bh) * a.T + (int64_t)c * L + t;
            a.fk[at] = f;
            a.dj[at] = g;
        }
    }
    if (a.dh0 && on) {
#pragma unroll
        for (int t = 0; t < NTL; ++t)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
                st4(a.dh0 + (bh * P + p0 + pw + ct * 16 + l16) * N + t * 16 + 4 * q, acc[t][ct]);
    }
}

// ---------------------------------------------------------------------------
// k_delta_grad: dB and dC of one chunk, group and slab of NS key columns, summed over a share
// of the group's heads in registers (and dbeta, by the first slab).  Wave w owns token tile
// w as the COLUMNS of dQ^T[n][i] and dK^T[n][i], so the 64 x 64 gradient tables it needs,
// dP^T and the two sides of W, come out of the matrix cores in the layout their products
// read.  Rows pass through LDS 32 headdim columns at a time, asked for a step ahead.  2 rows of
// 2048 tokens, 48 heads of 64, dstate 128, one group: 106 us for 0.26 GB (0.05 ms at copy rate;
// every wave fetching its own fragments took 171).  Everything here ends in the problem dtype: the states enter with one bfloat16
// term, r, z and the tables with two, so that every product has one rounded factor at most.
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ typename V8<T>::type bld8(brsrc r, int vo, int so) {
    const u32x4v a = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(r, vo, so, 0));
    if constexpr (sizeof(T) == 2) {
        return __builtin_bit_cast(bf16x8, a);
    } else {
        const u32x4v b = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(r, vo + 16, so, 0));
        return join(__builtin_bit_cast(f32x4, a), __builtin_bit_cast(f32x4, b));
    }
}

template <typename T, int N>
struct GradCfg {
    static constexpr int NS = N < 64 ? N : 64;
    static constexpr int LDN = NS + 8, LDP = 32 + 8;
    static constexpr int TILES = kTerms<T> > 1 ? 5 : 3;  // dY, r, z, and (bfloat16) the terms that r and z leave
    static constexpr size_t BYTES = (size_t)((2 * L + 2 * 32) * LDN + TILES * L * LDP) * sizeof(T) + (size_t)5 * L * 4;
};

template <typename T, int N>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void k_delta_grad(Args a) {
    typedef GradCfg<T, N> CF;
    constexpr int NS = CF::NS, LDN = CF::LDN, LDP = CF::LDP, NTL = NS / 16, SLABS = N / NS, TILES = CF::TILES;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), l16 = lane & 15, q = lane >> 4;
    const int H = a.H, G = a.G, P = a.P, KP = (P + 31) / 32;
    T* Ks = reinterpret_cast<T*>(smem);
    T* Qs = Ks + L * LDN;
    T* Hs = Qs + L * LDN;
    T* Ls = Hs + 32 * LDN;
    T* Ts = Ls + 32 * LDN;
    float* ecs = reinterpret_cast<float*>(Ts + TILES * L * LDP);
    float* ews = ecs + L;
    float* chi = ews + L;
    float* clo = chi + L;
    float* bts = clo + L;

    unsigned id = xcd_range(blockIdx.x, gridDim.x);
    const int slab = (int)(id % SLABS);
    id /= SLABS;
    const int sub = (int)(id % (unsigned)a.nsub);
    id /= (unsigned)a.nsub;
    const int g = (int)(id % (unsigned)G), kk = (int)(id / (unsigned)G);
    const int row = a.rows.row_of(kk), c = kk - a.rows.kbase(row);
    const int64_t t0 = a.rows.tok0(row) + (int64_t)c * L;
    const int n = (int)min((int64_t)L, a.rows.len(row) - (int64_t)c * L);
    const int Hg = H / G, per = (Hg + a.nsub - 1) / a.nsub;
    const int hb = g * Hg + sub * per, he = min(g * Hg + Hg, hb + per);
    const int n0 = slab * NS;

    // 32 headdim columns of a head at a time, asked for a step ahead
    typedef typename V8<T>::type F8;
    auto rows = [&](const void* p) {
        return make_rsrc(static_cast<const T*>(p) + t0 * H * P, (uint32_t)((int64_t)n * H * P * sizeof(T)));
    };
    auto states = [&](const void* p) {
        return make_rsrc(static_cast<const T*>(p) + (int64_t)kk * H * P * N, (uint32_t)((int64_t)H * P * N * sizeof(T)));
    };
    const brsrc src[5] = {rows(a.dy), rows(a.r), rows(a.z), rows(TILES > 3 ? a.rlo : a.r), rows(TILES > 3 ? a.zlo : a.z)};
    const brsrc hsrc = states(a.hin), lsrc = states(a.lin);
    F8 tv[TILES], hv, lv;
    float fv[5];
    const int tr = tid >> 2, tc = (tid & 3) << 3, hr = tid / (NS / 8), hc = (tid % (NS / 8)) << 3;
    constexpr int NONE = 0x7fff0000;  // beyond every resource: reads as zero
    const int to = tc < P ? (tr * H * P + tc) * (int)sizeof(T) : NONE;
    const int ho = hr < 32 && hr < P ? (hr * N + n0 + hc) * (int)sizeof(T) : NONE;
    auto load = [&](int h, int ks) {
        const int64_t e = (int64_t)kk * H + h;
        const int ts = (h * P + ks * 32) * (int)sizeof(T), hs = (h * P + ks * 32) * N * (int)sizeof(T);
#pragma unroll
        for (int k = 0; k < TILES; ++k) tv[k] = bld8<T>(src[k], to, ts);
        hv = bld8<T>(hsrc, ho, hs);
        lv = bld8<T>(lsrc, ho, hs);
        if (ks == 0 && tid < L) {
            fv[0] = a.vec[e * kVec + tid];
            fv[1] = a.vec[e * kVec + L + tid];
            fv[2] = a.vec[e * kVec + 3 * L + tid];
            fv[3] = a.vec[e * kVec + 4 * L + tid];
            fv[4] = tid < n ? to_f(static_cast<const T*>(a.beta)[(t0 + tid) * H + h]) : 0.f;
        }
    };
    auto put = [&](int ks) {
#pragma unroll
        for (int k = 0; k < TILES; ++k) st8(Ts + (k * L + tr) * LDP + tc, tv[k]);
        if (hr < 32) {
            st8(Hs + hr * LDN + hc, hv);
            st8(Ls + hr * LDN + hc, lv);
        }
        if (ks == 0 && tid < L)
#pragma unroll
            for (int k = 0; k < 5; ++k) ecs[k * L + tid] = fv[k];
    };
    if (hb < he) load(hb, 0);
    stage_rows(static_cast<const T*>(a.B) + (t0 * G + g) * N + n0, (int64_t)G * N, Ks, LDN, n, NS, NS, tid, 256);
    stage_rows(static_cast<const T*>(a.C) + (t0 * G + g) * N + n0, (int64_t)G * N, Qs, LDN, n, NS, NS, tid, 256);
    f32x4 dq[NTL], dk[NTL];
#pragma unroll
    for (int t = 0; t < NTL; ++t) dq[t] = dk[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int i = w * 16 + l16;  // this lane's token column

    for (int h = hb; h < he; ++h) {
        // r and z in two terms (the gradients of B would lose half of their rounding's room to
        // one): the product with a tensor that has one term, and of the two
        constexpr bool TWO = kTerms<T> > 1;
        // tables, rows j: pa = dP_{ij}, wa = W_{ij} in the tiles j <= i (i is this wave's), and in
        // those beyond dP_{ji}, W_{ji}; pd, wd the latter in the diagonal tile
        f32x4 pa[4], wa[4], pd = f32x4{0.f, 0.f, 0.f, 0.f}, wd = pd;
#pragma unroll
        for (int j = 0; j < 4; ++j) pa[j] = wa[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        f32x4 th[NTL], tz[NTL], tl[NTL];  // h^T dY^T, h^T z^T, dh'^T r^T
#pragma unroll
        for (int t = 0; t < NTL; ++t) th[t] = tz[t] = tl[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int ks = 0; ks < KP; ++ks) {
            wave_meet(false);  // the step before is done with its tiles
            put(ks);
            wave_meet(false);
            if (ks + 1 < KP) load(h, ks + 1);
            else if (h + 1 < he) load(h + 1, 0);
            auto rowf = [&](int k, int tile) { return ld8(Ts + (k * L + tile * 16 + l16) * LDP + 8 * q); };
            const F8 yi = rowf(0, w), ri = rowf(1, w), zi = rowf(2, w);
            F8 rl = ri, zl = zi;
            if (TWO) {
                rl = rowf(3, w);
                zl = rowf(4, w);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j <= w) {
                    const F8 rj = rowf(1, j);
                    pa[j] = mma(pa[j], rj, yi);
                    wa[j] = mma(wa[j], rj, zi);
                    if (TWO) {
                        const F8 rk = rowf(3, j);
                        pa[j] = mma(pa[j], rk, yi);
                        wa[j] = mma(wa[j], rk, zi);
                        wa[j] = mma(wa[j], rj, zl);
                    }
                } else {
                    const F8 yj = rowf(0, j), zj = rowf(2, j);
                    pa[j] = mma(pa[j], yj, ri);
                    wa[j] = mma(wa[j], zj, ri);
                    if (TWO) {
                        pa[j] = mma(pa[j], yj, rl);
                        wa[j] = mma(wa[j], zj, rl);
                        wa[j] = mma(wa[j], rowf(4, j), ri);
                    }
                }
            }
            pd = mma(pd, yi, ri);
            wd = mma(wd, zi, ri);
            if (TWO) {
                pd = mma(pd, yi, rl);
                wd = mma(wd, zi, rl);
                wd = mma(wd, zl, ri);
            }
#pragma unroll
            for (int t = 0; t < NTL; ++t) {
                const auto hf = frag_rows(Hs, LDN, 0, t * 16, lane);
                const auto lf = frag_rows(Ls, LDN, 0, t * 16, lane);
                th[t] = mma(th[t], hf, yi);
                tz[t] = mma(tz[t], hf, zi);
                tl[t] = mma(tl[t], lf, ri);
                if (TWO) {
                    tz[t] = mma(tz[t], hf, zl);
                    tl[t] = mma(tl[t], lf, rl);
                }
            }
        }
        const float bi = bts[i], ci = chi[i], di = clo[i];
        const float s1 = ecs[i], s2 = ecs[i] * bi, s3 = ews[i] * bi;
#pragma unroll
        for (int t = 0; t < NTL; ++t) {
            dq[t] += th[t] * s1;
            dk[t] += tl[t] * s3 - tz[t] * s2;
        }
        Sp<T> sp[2], sc[2], sw[2];  // dP below, dP above, W, with their decays
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            f32x4 pl[2], pu[2], wt[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int j = 2 * t + u;
                const f32x4 bo = ld4(bts + j * 16 + 4 * q), co = ld4(chi + j * 16 + 4 * q), lo = ld4(clo + j * 16 + 4 * q);
                if (j == w && slab == 0) {  // z_i . r_i sits on the diagonal of this wave's own tile
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (4 * q + r == l16 && i < n)
                            static_cast<T*>(a.dbeta)[(t0 + i) * H + h] = from_f<T>(wa[j][r]);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int o = j * 16 + 4 * q + r;  // the other token
                    const float d = (ci - co[r]) + (di - lo[r]);
                    const float e = exp2f_fast(o <= i ? d : -d);  // (above 1 where dt A > 0)
                    const bool up = j == w && o >= i;
                    pl[u][r] = o <= i ? pa[j][r] * (e * bo[r]) : 0.f;
                    pu[u][r] = o >= i ? (up ? pd[r] : pa[j][r]) * (e * bi) : 0.f;
                    wt[u][r] = o != i ? -(up ? wd[r] : wa[j][r]) * (e * bo[r] * bi) : 0.f;
                }
            }
            split8(join(pl[0], pl[1]), sp[t]);
            split8(join(pu[0], pu[1]), sc[t]);
            split8(join(wt[0], wt[1]), sw[t]);
        }
#pragma unroll
        for (int t = 0; t < NTL; ++t)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const auto kf = frag_rows_split(Ks, LDN, ks * 32 + 4 * q, ks * 32 + 16 + 4 * q, t * 16, lane);
                dk[t] = mma_es<2>(dk[t], kf, sw[ks]);
                if (2 * ks <= w) dq[t] = mma_es<2>(dq[t], kf, sp[ks]);
                if (2 * ks + 1 >= w) {
                    const auto qf = frag_rows_split(Qs, LDN, ks * 32 + 4 * q, ks * 32 + 16 + 4 * q, t * 16, lane);
                    dk[t] = mma_es<2>(dk[t], qf, sc[ks]);
                }
            }
    }
    if (i >= n) return;
    const int64_t o = ((t0 + i) * G + g) * N + n0 + 4 * q;
    if (a.nsub == 1) {
#pragma unroll
        for (int t = 0; t < NTL; ++t) {
            typename V4<T>::type ok, oq;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                ok[r] = from_f<T>(dk[t][r]);
                oq[r] = from_f<T>(dq[t][r]);
            }
            st4(static_cast<T*>(a.dB) + o + t * 16, ok);
            st4(static_cast<T*>(a.dC) + o + t * 16, oq);
        }
    } else {
        const int64_t all = (int64_t)a.rows.nrows * a.T * G * N;
        float* pk = a.part + (int64_t)sub * 2 * all + o;
#pragma unroll
        for (int t = 0; t < NTL; ++t) {
            st4(pk + t * 16, dk[t]);
            st4(pk + all + t * 16, dq[t]);
        }
    }
}

// dB and dC from the shares' partial sums, in share order
template <typename T>
__global__ __launch_bounds__(256) void k_delta_sum(const float* __restrict__ part, T* __restrict__ dB,
                                                   T* __restrict__ dC, int64_t all, int nsub) {
    const int64_t v = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (v >= 2 * all) return;
    f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < nsub; ++k) s += ld4(part + (int64_t)k * 2 * all + v);
    typename V4<T>::type o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = from_f<T>(s[e]);
    st4(v < all ? dB + v : dC + (v - all), o);
}

// ---------------------------------------------------------------------------
// k_delta_ddt: ddt of a chunk, and its share of dA, for `heads` heads of a group.  Wave w forms
// E_ij of its token tile (i, columns) with the tiles j <= w: Q K^T and K K^T once for all heads,
// dY r^T and z r^T per head, r and z in all their terms (two would leave ddt ten times its error).
// The sum over the pairs around each token t is taken as it stands, never as a difference of
// longer sums: pairs of a later tile's i by their j, summed over the earlier tokens at the end; the
// tile's own by a product with ones below the diagonal (j < t) and a mask (i >= t).  The rest are
// sums along the chunk, one token per lane, in float64.
// Rows are fetched straight into LDS, W headdim columns (8 elements at a time exchanged by the
// row's low bits), a head's while the sums of the one before are formed.  Bound by the latency of
// these steps, two work-groups a CU: 2 rows of 2048 tokens, 48 heads of 64, dstate 128: 65 us, 35 for
// its 0.18 GB at the copy rate.
// ---------------------------------------------------------------------------
// a 64 x W tile of rows `stride` bytes apart: instruction `m` of TileW<T, W>::RUNS
template <typename T, int W>
struct TileW {
    static constexpr int ELEMS = L * W, RUNS = ELEMS * (int)sizeof(T) / 1024, BLOCKS = W / 8;
    static __device__ __forceinline__ void fetch(brsrc r, T* dst, int stride, int so, int m, int lane) {
        const int o = (m * 1024 + lane * 16) / (int)sizeof(T), row = o / W, col = o % W;
        const int src = ((col >> 3) ^ (row & (BLOCKS - 1))) * 8 + (col & 7);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(dst + m * (1024 / (int)sizeof(T))), 16,
                                                 row * stride + src * (int)sizeof(T), so, 0, 0);
    }
    // operand of rows `row`, columns 32 k + 8 q on (past W: zero)
    static __device__ __forceinline__ typename V8<T>::type frag(const T* tile, int row, int k, int q) {
        const int b = 4 * k + q;
        return sel8(W >= 32 || b < BLOCKS, ld8(tile + row * W + (((b & (BLOCKS - 1)) ^ (row & (BLOCKS - 1))) << 3)));
    }
};
template <typename T, int W>
struct DdtCfg {
    static constexpr int TILES = 1 + 2 * kTerms<T>;  // dY, r, z
    static constexpr int KEYS = 4 * L * 64;          // elements of two K and Q tiles (bfloat16; float32: one of each)
    static constexpr int ROWS = TILES * TileW<T, W>::ELEMS;
    static constexpr int ELEMS = ROWS > KEYS / (int)(sizeof(T) / 2) ? ROWS : KEYS / (int)(sizeof(T) / 2);
};

template <typename T, int W>
__global__ __launch_bounds__(256, 2) void k_delta_ddt(Args a, int heads) {
    constexpr int NT = kTerms<T>;
    typedef TileW<T, W> TW;
    typedef typename V8<T>::type F8;
    __shared__ __attribute__((aligned(16))) T buf[DdtCfg<T, W>::ELEMS];
    __shared__ __attribute__((aligned(16))) float pairs[2][4][L];
    const int lane = threadIdx.x & 63, w = wave_id(), l16 = lane & 15, q = lane >> 4;
    const int H = a.H, G = a.G, P = a.P, N = a.N, Hg = H / G, nhb = (Hg + heads - 1) / heads;
    unsigned id = xcd_range(blockIdx.x, gridDim.x);
    const int hb = (int)(id % (unsigned)nhb);
    id /= (unsigned)nhb;
    const int g = (int)(id % (unsigned)G), kk = (int)(id / (unsigned)G);
    const int row = kk / a.nc, c = kk - row * a.nc, BH = a.rows.nrows * H;
    const int64_t t0 = (int64_t)row * a.T + (int64_t)c * L;
    const int n = (int)min((int64_t)L, a.T - (int64_t)c * L);
    const int i = w * 16 + l16;
    constexpr int ES = (int)sizeof(T);

    // (rows past the end read as zero)
    const int rsx = H * P * ES, rsk = G * N * ES;
    auto keys = [&](const void* p) {
        return make_rsrc(static_cast<const T*>(p) + (t0 * G + g) * N, (uint32_t)((n - 1) * rsk + N * ES));
    };
    f32x4 qk[4], kd[4];  // Q_i . K_j, K_i . K_j: rows j, column i
#pragma unroll
    for (int j = 0; j < 4; ++j) qk[j] = kd[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    {
        const brsrc kr = keys(a.B), qr = keys(a.C);
        // PAIRS K and Q tiles of KW columns from column k0 on
        auto products = [&](int k0, auto kw, auto np) {
            constexpr int KW = decltype(kw)::value, NP = decltype(np)::value;
            typedef TileW<T, KW> TK;
            wave_meet(false);  // the tiles before are no longer read
            for (int m = w; m < NP * 2 * TK::RUNS; m += 4) {
                const int tile = m / TK::RUNS;
                TK::fetch(tile & 1 ? qr : kr, buf + tile * TK::ELEMS, rsk, (k0 + (tile >> 1) * KW) * ES, m % TK::RUNS, lane);
            }
            wave_meet(true);
#pragma unroll
            for (int u = 0; u < NP; ++u)
#pragma unroll
                for (int k = 0; k < (KW + 31) / 32; ++k) {
                    const T *kt = buf + 2 * u * TK::ELEMS, *qt = kt + TK::ELEMS;
                    const F8 qi = TK::frag(qt, i, k, q), ki = TK::frag(kt, i, k, q);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j <= w) {
                            const F8 kj = TK::frag(kt, j * 16 + l16, k, q);
                            qk[j] = mma(qk[j], kj, qi);
                            kd[j] = mma(kd[j], kj, ki);
                        }
                }
        };
        const std::integral_constant<int, 1> one;
        const std::integral_constant<int, 64> k64;
        if (N == 16) products(0, std::integral_constant<int, 16>(), one);
        else if (N == 32) products(0, std::integral_constant<int, 32>(), one);
        else if (NT == 1 || N == 64)
            for (int k0 = 0; k0 < N; k0 += 64) products(k0, k64, one);
        else if constexpr (NT > 1)
            for (int k0 = 0; k0 < N; k0 += 128) products(k0, k64, std::integral_constant<int, 2>());
    }
    auto fetch = [&](int h, int k0) {
        for (int m = w; m < DdtCfg<T, W>::TILES * TW::RUNS; m += 4) {
            const int tile = m / TW::RUNS;
            const void* p = tile == 0 ? a.dy : tile == 1 ? a.r : tile == 2 ? a.z : tile == 3 ? a.rlo
                            : tile == 4 ? a.zlo : tile == 5 ? a.rll : a.zll;
            const brsrc r = make_rsrc(static_cast<const T*>(p) + t0 * H * P, (uint32_t)(n * rsx));
            TW::fetch(r, buf + tile * TW::ELEMS, rsx, (h * P + k0) * ES, m % TW::RUNS, lane);
        }
    };

    const int h0 = g * Hg + hb * heads, h1 = min(g * Hg + Hg, h0 + heads);
    wave_meet(false);  // the key tiles are no longer read
    fetch(h0, 0);
    for (int h = h0; h < h1; ++h) {
        const int64_t e = (int64_t)kk * H + h;
        const float* vec = a.vec + e * kVec;
        f32x4 pa[4], wa[4];  // dY_i . r_j, z_i . r_j
#pragma unroll
        for (int j = 0; j < 4; ++j) pa[j] = wa[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        // (asked for before the next tiles are: loads return in order)
        const float bi = vec[2 * L + i], ci = vec[3 * L + i], di = vec[4 * L + i];
        f32x4 bo[4], co[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= w) {
                const float* vj = vec + j * 16 + 4 * q;
                bo[j] = ld4(vj + 2 * L);
                co[j] = ld4(vj + 3 * L);
                lo[j] = ld4(vj + 4 * L);
            }
        // one wave finishes the head; its sums along the chunk, while the tiles come
        const bool last = w == ((h - h0) & 3), on = lane < n;
        const int64_t to = (t0 + (on ? lane : 0)) * H + h;
        double v = 0.0, dtv = 0.0;
        if (last) {
            const int64_t at = ((int64_t)row * H + h) * a.T + (int64_t)c * L + lane;
            double f = 0.0, d = 0.0;
            if (lane < a.tots) v = (double)a.tot[(int64_t)lane * a.ntab * H + e];
            dtv = (double)a.dt[to];
            for (int s0 = 0; s0 < a.slices; s0 += 4) {  // (a load that waits for the one before costs 1 us)
                float x[4], y[4], z[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t o = (int64_t)min(s0 + k, a.slices - 1) * BH * a.T + (on ? at : at - lane);
                    x[k] = a.fq[o];
                    y[k] = a.fk[o];
                    z[k] = a.dj[o];
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (on && s0 + k < a.slices) {
                        f += (double)x[k] - (double)y[k];
                        d += (double)z[k];
                    }
            }
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
            d = __shfl_up(d, 1, 64);
            if (lane == 0) d = 0.0;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const double o = __shfl_down(f, off, 64), p = __shfl_up(d, off, 64);
                if (lane + off < 64) f += o;
                if (lane >= off) d += p;
            }
            v += f + d;
        }
        for (int k0 = 0; k0 < P; k0 += W) {
            wave_meet(true);  // the tiles have landed
            auto tile = [&](int k) { return buf + k * TW::ELEMS; };  // dY, r, z, then the further terms of r and z
#pragma unroll
            for (int k = 0; k < (W + 31) / 32; ++k) {
                const F8 yi = TW::frag(tile(0), i, k, q);
                F8 zi[NT];
#pragma unroll
                for (int m = 0; m < NT; ++m) zi[m] = TW::frag(tile(2 + 2 * m), i, k, q);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j <= w)
#pragma unroll
                        for (int m = 0; m < NT; ++m) {
                            const F8 rj = TW::frag(tile(1 + 2 * m), j * 16 + l16, k, q);
                            pa[j] = mma(pa[j], rj, yi);
#pragma unroll
                            for (int o = 0; o < NT - m; ++o) wa[j] = mma(wa[j], rj, zi[o]);
                        }
            }
            wave_meet(false);  // and are no longer read
            if (k0 + W < P) fetch(h, k0 + W);
            else if (h + 1 < h1) fetch(h + 1, 0);
        }
        float(*pr)[L] = pairs[(h - h0) & 1];
        // of four rows' sums, that of this lane's row
        auto own_row = [&](f32x4 v) {
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = row_sum16(v[r]);
            return l16 & 2 ? (l16 & 1 ? v[3] : v[2]) : (l16 & 1 ? v[1] : v[0]);
        };
        f32x4 es = f32x4{0.f, 0.f, 0.f, 0.f}, ed = es;  // E of the tiles before w, added up; of the diagonal tile
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= w) {
                f32x4 ev;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float gam = exp2f_fast((ci - co[j][r]) + (di - lo[j][r]));
                    ev[r] = j < w || 4 * q + r < l16 ? gam * bo[j][r] * (pa[j][r] * qk[j][r] - bi * wa[j][r] * kd[j][r]) : 0.f;
                }
                if (j == w) {
                    ed = ev;
                } else {
                    es += ev;
                    const float s = own_row(ev);
                    if (l16 < 4) pr[w][j * 16 + 4 * q + l16] = s;
                }
            }
        const f32x4 one = f32x4{1.f, 1.f, 1.f, 1.f};
        f32x4 below, m;
#pragma unroll
        for (int r = 0; r < 4; ++r) below[r] = 4 * q + r < l16 ? 1.f : 0.f;
        m = mma16(mma16(f32x4{0.f, 0.f, 0.f, 0.f}, one, es), below, ed);
#pragma unroll
        for (int r = 0; r < 4; ++r) m[r] = l16 >= 4 * q + r ? m[r] : 0.f;
        const float s = own_row(m);
        if (l16 < 4) pr[w][w * 16 + 4 * q + l16] = s;
        wave_meet(false);
        if (!last) continue;
        // the pairs by j: within its tile over the tokens before this one, and the tiles before
        // (sums of 16 in float32)
        const float c1 = lane < 16 ? pr[1][lane] : 0.f, c2 = lane < 32 ? pr[2][lane] : 0.f, c3 = lane < 48 ? pr[3][lane] : 0.f;
        float x = c1 + c2 + c3;
        const float s2 = row_sum16(c2), s3 = row_sum16(c3);
        x = row_shift<1>(x);
        x += row_shift<1>(x);
        x += row_shift<2>(x);
        x += row_shift<4>(x);
        x += row_shift<8>(x);
        const float s20 = __shfl(s2, 0, 64), s30 = __shfl(s3, 0, 64), s31 = __shfl(s3, 16, 64);
        v += (double)pr[lane >> 4][lane] + (double)x;
        if ((lane >> 4) == 1) v += (double)s20 + (double)s30;
        if ((lane >> 4) == 2) v += (double)s30 + (double)s31;
        if (on) a.ddt[to] = (float)(v * (double)a.A[h]);
        double da = on ? v * dtv : 0.0;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) da += __shfl_xor(da, off, 64);
        if (lane == 0) a.dAp[e] = da;
    }
}
// dA_h over the chunks, in order
template <int BLOCK = 64>
__global__ __launch_bounds__(BLOCK) void k_delta_dA(const double* __restrict__ p, float* __restrict__ dA, int ntab,
                                                    int H) {
    const int h = blockIdx.x;
    double s = 0.0;
    for (int v = threadIdx.x; v < ntab; v += BLOCK) s += p[(int64_t)v * H + h];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
    if (threadIdx.x == 0) dA[h] = (float)s;
}

// ---------------------------------------------------------------------------
// k_delta_step: the recurrence token by token on a held state, in place, all in float32.
// One thread owns 8 consecutive elements of a state row p; the N / 8 lanes of a row (one
// wave) reduce h B and then h C.  The state is read and written once per call: bound by HBM.
// 64 rows, 80 heads of 64, dstate 128: 66 us for 0.34 GB, 5.1 TB/s, what a copy reaches (51 us where the
// state is still in the last-level cache from the call before).  One row of 32
// heads of 128: 4 us, behind 10 us of the host's.
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(256) void k_delta_step(const T* __restrict__ x, const float* __restrict__ dt,
                                                    const float* __restrict__ A, const T* __restrict__ Bm,
                                                    const T* __restrict__ Cm, const T* __restrict__ beta,
                                                    float* __restrict__ hst, T* __restrict__ y, int64_t Tn, int H,
                                                    int P, int N, int G) {
    constexpr int E = 8;
    const int64_t bh = blockIdx.x;
    const int h = (int)(bh % H), g = h / (H / G);
    const int64_t bi = bh / H;
    const int e0 = (blockIdx.y * 256 + threadIdx.x) * E;
    const bool active = e0 < P * N;
    const int ec = active ? e0 : 0, p = ec / N, n0 = ec % N, R = N / E, lane = threadIdx.x & 63;
    float* hp = hst + bh * (int64_t)P * N + ec;
    float hv[E];
#pragma unroll
    for (int k = 0; k < E; ++k) hv[k] = 0.f;
    if (active) {
        const f32x8 v = ld8(hp);
#pragma unroll
        for (int k = 0; k < E; ++k) hv[k] = v[k];
    }
    const double Ah = (double)A[h] * 1.4426950408889634;
    for (int64_t t = 0; t < Tn; ++t) {
        const int64_t row = bi * Tn + t;
        const float d = exp2f_fast((float)((double)dt[row * H + h] * Ah));
        const float xp = to_f(x[(row * H + h) * P + p]), bt = to_f(beta[row * H + h]);
        float bv[E], cv[E], s = 0.f, o = 0.f;
        const T* br = Bm + (row * G + g) * N + n0;
        const T* cr = Cm + (row * G + g) * N + n0;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            bv[k] = to_f(br[k]);
            cv[k] = to_f(cr[k]);
        }
#pragma unroll
        for (int k = 0; k < E; ++k) {
            hv[k] *= d;
            s += hv[k] * bv[k];
        }
        for (int off = R >> 1; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
        const float u = bt * (xp - s);
#pragma unroll
        for (int k = 0; k < E; ++k) {
            hv[k] += u * bv[k];
            o += hv[k] * cv[k];
        }
        for (int off = R >> 1; off > 0; off >>= 1) o += __shfl_xor(o, off, 64);
        if (active && (lane & (R - 1)) == 0) y[(row * H + h) * P + p] = from_f<T>(o);
    }
    if (active) {
        f32x8 v;
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = hv[k];
        st8(hp, v);
    }
}

}  // namespace delta
}  // namespace ssd
