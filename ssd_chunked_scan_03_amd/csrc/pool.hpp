// pool.hpp -- states of many sequences in the slots of a pool: the recurrence through slot
// indices, one token after another or along the accepted path of a tree.
#pragma once

#include "delta.hpp"
#include "device.hpp"

namespace ssd {
namespace pool {

constexpr int kNodes = 256;  // nodes of a tree at most

struct Args {
    int64_t b, T;  // rows, tokens (nodes) of a row
    int H, P, N, G;
    int64_t xs, bs, cs;  // elements between tokens of x, B, C
    int64_t S, ss;       // slots of the pool, elements between them
    const void* x;
    const float* dt;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    const void* beta;  // nullptr: the scan's recurrence
    const int* parents;
    const int* last;
    float* pool;
    const int* slots;
    const int* out;  // never nullptr
    void* y;
    hipStream_t stream;
};

// ---------------------------------------------------------------------------
// k_walk: h <- a h + u B^T (u = x, or beta (x - a h B) for the delta rule) over a row's tokens, or
// (PATH) over the nodes from the held state to node last[i], all in float32.  A thread owns CH times 8
// consecutive elements of state rows, 2048 elements apart; the N / 8 lanes of a row reduce h B and h C.  The
// state is read once and written once, and asked for first.  Tokens' operands (STAGE) come to LDS
// kBatch tokens at a time, so that their latency is paid once for all of them; a single token's
// go straight to registers.  Grid (b H, ceil(P N / (2048 CH))), 256 threads.
// Bound by the state's bytes where there are many rows: one token of 128 rows, 80 heads of 64, dstate 128, 671 MB in 136 us
// (4.9 TB/s; a large copy reaches 5.2); paths of 5 nodes of 64 such rows with the delta rule, 336 MB, 78 us, behind the
// walk up the tree and the row sums of every token.  One row of 48 heads: 5 us, a chain of latencies.  Deep paths are
// bound by the vector operations of one token after another: 100 nodes of 16 rows, 32 heads of 64, dstate 256, 67 MB of
// states, 70 us, the delta rule 127 (float32 246).
// ---------------------------------------------------------------------------
constexpr int kBatch = 16;

// The sum over R = 2 .. 32 neighbouring lanes, in each of them: inside a row of 16 in the ALU (through LDS the
// commit of 64 rows below takes 81 us, so 78).
__device__ __forceinline__ float lanes_sum(float v, int R) {
    v += delta::lane_turn<0xB1>(v);            // lane ^ 1
    if (R > 2) v += delta::lane_turn<0x4E>(v);   // lane ^ 2
    if (R > 4) v += delta::lane_turn<0x141>(v);  // the other four of eight, mirrored
    if (R > 8) v += delta::lane_turn<0x140>(v);  // the other eight of sixteen, mirrored
    if (R > 16) v += __shfl_xor(v, 16, 64);
    return v;
}

template <typename T, bool DELTA, bool PATH, bool STAGE, int CH>
__global__ __launch_bounds__(256) void k_walk(Args a) {
    constexpr int E = 8, EV = 16 / (int)sizeof(T);
    extern __shared__ __attribute__((aligned(16))) char smem[];  // STAGE: B [kBatch][N], x [kBatch][P], C [kBatch][N]
    __shared__ int path[PATH ? kNodes : 1];
    __shared__ int par[PATH ? kNodes : 1];
    __shared__ float dec[STAGE ? kBatch : 1], bet[STAGE ? kBatch : 1];
    const int64_t bh = blockIdx.x;
    const int h = (int)(bh % a.H), g = h / (a.H / a.G), tid = threadIdx.x;
    const int64_t bi = bh / a.H;
    const int P = a.P, N = a.N;
    const int slot = a.slots[bi], out = a.out[bi];
    const bool live = slot >= 0 && slot < a.S, writes = live && out >= 0 && out < a.S;
    const int e0 = (blockIdx.y * CH * 256 + tid) * E;
    const bool active = e0 < P * N;  // (CH > 1 only where all are)
    const int ec = active ? e0 : 0, p = ec / N, n0 = ec % N, R = N / E, lane = tid & 63, dp = 2048 / N;
    float hv[CH][E];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        f32x8 v = {};
        if (active && live) v = ld8(a.pool + (int64_t)slot * a.ss + (int64_t)h * P * N + ec + c * 2048);
#pragma unroll
        for (int k = 0; k < E; ++k) hv[c][k] = v[k];
    }
    const T* x = static_cast<const T*>(a.x) + h * P;
    const T* Bm = static_cast<const T*>(a.B) + g * N;
    const T* Cm = static_cast<const T*>(a.C) + g * N;
    const T* beta = static_cast<const T*>(a.beta);
    T* y = static_cast<T*>(a.y);
    int64_t steps = a.T;
    if (PATH) {
        for (int k = tid; k < a.T; k += 256) par[k] = a.parents[bi * a.T + k];
        __syncthreads();
        // the nodes from last[i] up to the held state; a parent outside [-1, k) ends the row
        int k = a.last[bi], d = 0;
        bool there = k >= -1 && k < a.T;
        while (there && k >= 0) {
            if (tid == 0) path[d] = k;
            ++d;
            const int up = par[k];
            there = up >= -1 && up < k;
            k = up;
        }
        if (!there || !live) return;
        __syncthreads();
        steps = d;
    } else if (!live) {
        for (int64_t t = 0; t < a.T; ++t)
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (active && (lane & (R - 1)) == 0) y[((bi * a.T + t) * a.H + h) * P + p + c * dp] = from_f<T>(0.f);
        return;
    }
    const double Ah = (double)a.A[h] * 1.4426950408889634;
    const float Dh = !PATH && a.D ? a.D[h] : 0.f;
    auto token = [&](int64_t t) { return bi * a.T + (PATH ? path[steps - 1 - t] : t); };
    auto step = [&](int64_t row, float d, float bt, const T* br, const T* cr, const T* xr) {
        float bv[E], cv[E];
#pragma unroll
        for (int k = 0; k < E; ++k) {
            bv[k] = to_f(br[k]);
            if (!PATH) cv[k] = to_f(cr[k]);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const float xp = to_f(xr[c * dp]);
            float s = 0.f, o = 0.f, u = xp;
#pragma unroll
            for (int k = 0; k < E; ++k) hv[c][k] *= d;
            if (DELTA) {
#pragma unroll
                for (int k = 0; k < E; ++k) s += hv[c][k] * bv[k];
                s = lanes_sum(s, R);
                u = bt * (xp - s);
            }
#pragma unroll
            for (int k = 0; k < E; ++k) hv[c][k] += u * bv[k];
            if (!PATH) {
#pragma unroll
                for (int k = 0; k < E; ++k) o += hv[c][k] * cv[k];
                o = lanes_sum(o, R);
                if (active && (lane & (R - 1)) == 0) y[(row * a.H + h) * P + p + c * dp] = from_f<T>(o + Dh * xp);
            }
        }
    };
    auto decay = [&](int64_t row) { return exp2f_fast((float)((double)a.dt[row * a.H + h] * Ah)); };
    if (!STAGE) {
        for (int64_t t = 0; t < steps; ++t) {
            const int64_t row = token(t);
            step(row, decay(row), DELTA ? to_f(beta[row * a.H + h]) : 0.f, Bm + row * a.bs + n0, Cm + row * a.cs + n0,
                 x + row * a.xs + p);
        }
    } else {
        T* sb = reinterpret_cast<T*>(smem);
        T* sx = sb + kBatch * N;
        T* sc = sx + kBatch * P;
        const int nv = N / EV, pv = P / EV;  // 16-byte pieces of a row of B, of x
        for (int64_t t0 = 0; t0 < steps; t0 += kBatch) {
            const int n = steps - t0 < kBatch ? (int)(steps - t0) : kBatch;
            if (t0 > 0) __syncthreads();
            if (tid < n) {
                const int64_t row = token(t0 + tid);
                dec[tid] = decay(row);
                if (DELTA) bet[tid] = to_f(beta[row * a.H + h]);
            }
            for (int i = tid; i < n * nv; i += 256) {
                const int t = i / nv, k = i % nv * EV;
                const int64_t row = token(t0 + t);
                *reinterpret_cast<f32x4*>(sb + t * N + k) = *reinterpret_cast<const f32x4*>(Bm + row * a.bs + k);
                if (!PATH) *reinterpret_cast<f32x4*>(sc + t * N + k) = *reinterpret_cast<const f32x4*>(Cm + row * a.cs + k);
            }
            for (int i = tid; i < n * pv; i += 256) {
                const int t = i / pv, k = i % pv * EV;
                *reinterpret_cast<f32x4*>(sx + t * P + k) = *reinterpret_cast<const f32x4*>(x + token(t0 + t) * a.xs + k);
            }
            __syncthreads();
            for (int t = 0; t < n; ++t)
                step(bi * a.T + t0 + t, dec[t], DELTA ? bet[t] : 0.f, sb + t * N + n0, sc + t * N + n0, sx + t * P + p);
        }
    }
    if (active && writes) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            f32x8 v;
#pragma unroll
            for (int k = 0; k < E; ++k) v[k] = hv[c][k];
            st8(a.pool + (int64_t)out * a.ss + (int64_t)h * P * N + ec + c * 2048, v);
        }
    }
}

template <typename T, bool DELTA, bool PATH, bool STAGE, int CH>
int launch_walk(const Args& a) {
    const size_t lds = STAGE ? (size_t)kBatch * (a.P + (PATH ? 1 : 2) * a.N) * sizeof(T) : 0;
    const dim3 grid((unsigned)(a.b * a.H), (unsigned)((a.P * a.N + 2048 * CH - 1) / (2048 * CH)));
    k_walk<T, DELTA, PATH, STAGE, CH><<<grid, 256, lds, a.stream>>>(a);
    return hipGetLastError() == hipSuccess ? 0 : 7;
}
template <typename T, bool DELTA, bool PATH, bool STAGE>
int walk_chunks(const Args& a, int ch) {
    if constexpr (!PATH) {
        if (ch == 4) return launch_walk<T, DELTA, PATH, STAGE, 4>(a);
    }
    if (ch == 2) return launch_walk<T, DELTA, PATH, STAGE, 2>(a);
    return launch_walk<T, DELTA, PATH, STAGE, 1>(a);
}
template <typename T, bool DELTA>
int walk_rule(const Args& a, bool path) {
    // The most state a thread that leaves every CU its eight work-groups, so that fewer work-groups read a token's
    // operands (8 / 16 / 32 elements a thread: one token of 128 rows, 80 heads of 64, dstate 128, 143 / 139 / 136 us; the
    // delta rule's commit of 64 such rows, paths of 5 nodes, 82 / 79 / 80 us).
    const int64_t pn = (int64_t)a.P * a.N, all = a.b * a.H;
    int ch = path ? 2 : 4;
    while (ch > 1 && (pn % (2048 * ch) != 0 || all * (pn / (2048 * ch)) < 2048)) ch >>= 1;
    if (path) return walk_chunks<T, DELTA, true, true>(a, ch);
    return a.T == 1 ? walk_chunks<T, DELTA, false, false>(a, ch) : walk_chunks<T, DELTA, false, true>(a, ch);
}
template <typename T>
int run_walk(const Args& a, bool path) { return a.beta ? walk_rule<T, true>(a, path) : walk_rule<T, false>(a, path); }

}  // namespace pool
}  // namespace ssd
