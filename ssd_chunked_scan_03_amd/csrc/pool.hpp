// pool.hpp -- states of many sequences in the slots of a pool: the recurrence through slot
// indices, one token after another or along the accepted path of a tree.
#pragma once

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
// (PATH) over the nodes from the held state to node last[i], all in float32.  One thread owns 8
// consecutive elements of a state row; the N / 8 lanes of a row reduce h B and h C.  Grid (b H,
// ceil(P N / 2048)), 256 threads.
// ---------------------------------------------------------------------------
template <typename T, bool DELTA, bool PATH>
__global__ __launch_bounds__(256) void k_walk(Args a) {
    constexpr int E = 8;
    __shared__ int path[PATH ? kNodes : 1];
    __shared__ int par[PATH ? kNodes : 1];
    const int64_t bh = blockIdx.x;
    const int h = (int)(bh % a.H), g = h / (a.H / a.G);
    const int64_t bi = bh / a.H;
    const int P = a.P, N = a.N;
    const int slot = a.slots[bi], out = a.out[bi];
    const bool live = slot >= 0 && slot < a.S, writes = live && out >= 0 && out < a.S;
    const int e0 = (blockIdx.y * 256 + threadIdx.x) * E;
    const bool active = e0 < P * N;
    const int ec = active ? e0 : 0, p = ec / N, n0 = ec % N, R = N / E, lane = threadIdx.x & 63;
    float hv[E];
#pragma unroll
    for (int k = 0; k < E; ++k) hv[k] = 0.f;
    if (active && live) {
        const f32x8 v = ld8(a.pool + (int64_t)slot * a.ss + (int64_t)h * P * N + ec);
#pragma unroll
        for (int k = 0; k < E; ++k) hv[k] = v[k];
    }
    const T* x = static_cast<const T*>(a.x);
    const T* Bm = static_cast<const T*>(a.B);
    const T* Cm = static_cast<const T*>(a.C);
    const T* beta = static_cast<const T*>(a.beta);
    T* y = static_cast<T*>(a.y);
    int64_t steps = a.T;
    if (PATH) {
        for (int k = threadIdx.x; k < a.T; k += 256) par[k] = a.parents[bi * a.T + k];
        __syncthreads();
        // the nodes from last[i] up to the held state; a parent outside [-1, k) ends the row
        int k = a.last[bi], d = 0;
        bool there = k >= -1 && k < a.T;
        while (there && k >= 0) {
            if (threadIdx.x == 0) path[d] = k;
            ++d;
            const int up = par[k];
            there = up >= -1 && up < k;
            k = up;
        }
        __syncthreads();
        if (!there || !live) return;
        steps = d;
    } else if (!live) {
        for (int64_t t = 0; t < a.T; ++t)
            if (active && (lane & (R - 1)) == 0) y[((bi * a.T + t) * a.H + h) * P + p] = from_f<T>(0.f);
        return;
    }
    const double Ah = (double)a.A[h] * 1.4426950408889634;
    const float Dh = !PATH && a.D ? a.D[h] : 0.f;
    for (int64_t t = 0; t < steps; ++t) {
        const int64_t row = bi * a.T + (PATH ? path[steps - 1 - t] : t);
        const float d = exp2f_fast((float)((double)a.dt[row * a.H + h] * Ah));
        const float xp = to_f(x[row * a.xs + h * P + p]);
        float bv[E], cv[E], s = 0.f, o = 0.f, u = xp;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            bv[k] = to_f(Bm[row * a.bs + g * N + n0 + k]);
            if (!PATH) cv[k] = to_f(Cm[row * a.cs + g * N + n0 + k]);
        }
#pragma unroll
        for (int k = 0; k < E; ++k) hv[k] *= d;
        if (DELTA) {
#pragma unroll
            for (int k = 0; k < E; ++k) s += hv[k] * bv[k];
            for (int off = R >> 1; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
            u = to_f(beta[row * a.H + h]) * (xp - s);
        }
#pragma unroll
        for (int k = 0; k < E; ++k) hv[k] += u * bv[k];
        if (!PATH) {
#pragma unroll
            for (int k = 0; k < E; ++k) o += hv[k] * cv[k];
            for (int off = R >> 1; off > 0; off >>= 1) o += __shfl_xor(o, off, 64);
            if (active && (lane & (R - 1)) == 0) y[(row * a.H + h) * P + p] = from_f<T>(o + Dh * xp);
        }
    }
    if (active && writes) {
        f32x8 v;
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = hv[k];
        st8(a.pool + (int64_t)out * a.ss + (int64_t)h * P * N + ec, v);
    }
}

template <typename T>
int run_walk(const Args& a, bool path) {
    const dim3 grid((unsigned)(a.b * a.H), (unsigned)((a.P * a.N + 2047) / 2048));
    if (path) {
        if (a.beta) k_walk<T, true, true><<<grid, 256, 0, a.stream>>>(a);
        else k_walk<T, false, true><<<grid, 256, 0, a.stream>>>(a);
    } else {
        if (a.beta) k_walk<T, true, false><<<grid, 256, 0, a.stream>>>(a);
        else k_walk<T, false, false><<<grid, 256, 0, a.stream>>>(a);
    }
    return hipGetLastError() == hipSuccess ? 0 : 7;
}

}  // namespace pool
}  // namespace ssd
