// tree.hpp -- a tree of drafted tokens over held states.  With E_k and W_kj the decays to node k
// along its path from the held state h and from node j:
//
//   u_k = x_k, or beta_k (x_k - E_k h B_k - sum_{j above k} W_kj (B_k . B_j) u_j)
//   y_k = E_k h C_k + sum_{j = k or above k} W_kj (C_k . B_j) u_j + D x_k
#pragma once

#include "pool.hpp"

namespace ssd {
namespace pool {

// One work-group per (row, head) takes the nodes in order: parts = 256 / P threads share a column p of
// the state, u stays in LDS, and every node walks up to its ancestors.
template <typename T, bool DELTA>
__global__ __launch_bounds__(256) void k_tree(Args a) {
    extern __shared__ __attribute__((aligned(16))) float u[];  // [T][P]
    __shared__ int par[kNodes], there[kNodes];
    const int64_t bh = blockIdx.x;
    const int h = (int)(bh % a.H), g = h / (a.H / a.G), P = a.P, N = a.N, K = (int)a.T;
    const int64_t bi = bh / a.H, row0 = bi * a.T;
    const int tid = threadIdx.x, parts = 256 / P, p = tid / parts, part = tid % parts;
    const int slot = a.slots[bi];
    const T* x = static_cast<const T*>(a.x) + row0 * a.xs + h * P;
    const T* Bm = static_cast<const T*>(a.B) + row0 * a.bs + g * N;
    const T* Cm = static_cast<const T*>(a.C) + row0 * a.cs + g * N;
    const T* beta = static_cast<const T*>(a.beta) + (DELTA ? row0 * a.H + h : 0);
    const float* dt = a.dt + row0 * a.H + h;
    T* y = static_cast<T*>(a.y) + (row0 * a.H + h) * P;
    const int64_t ys = (int64_t)a.H * P;
    if (slot < 0 || slot >= a.S) {
        for (int k = 0; k < K; ++k)
            if (part == 0) y[k * ys + p] = from_f<T>(0.f);
        return;
    }
    const float* hp = a.pool + slot * a.ss + (int64_t)(h * P + p) * N;
    for (int k = tid; k < K; k += 256) par[k] = a.parents[row0 + k];
    __syncthreads();
    if (tid == 0)
        for (int k = 0; k < K; ++k) there[k] = par[k] >= -1 && par[k] < k && (par[k] < 0 || there[par[k]]);
    __syncthreads();
    const double A = (double)a.A[h] * 1.4426950408889634;
    const float D = a.D ? a.D[h] : 0.f;
    auto sum = [&](float v) {
        for (int off = parts >> 1; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
        return v;
    };
    for (int k = 0; k < K; ++k) {
        if (!there[k]) {
            if (part == 0) y[k * ys + p] = from_f<T>(0.f);
            continue;
        }
        float v = 0.f, o = 0.f;
        for (int n = part; n < N; n += parts) {
            v += hp[n] * to_f(Bm[k * a.bs + n]);
            o += hp[n] * to_f(Cm[k * a.cs + n]);
        }
        v = sum(v);
        o = sum(o);
        double s = (double)dt[(int64_t)k * a.H] * A;
        float less = 0.f, more = 0.f;  // the ancestors' terms of u and of y
        for (int j = par[k]; j >= 0; j = par[j]) {
            const float w = exp2f_fast((float)s);
            float kk = 0.f, qk = 0.f;
            for (int n = part; n < N; n += parts) {
                const float b = to_f(Bm[j * a.bs + n]);
                kk += to_f(Bm[k * a.bs + n]) * b;
                qk += to_f(Cm[k * a.cs + n]) * b;
            }
            less += w * sum(kk) * u[j * P + p];
            more += w * sum(qk) * u[j * P + p];
            s += (double)dt[(int64_t)j * a.H] * A;
        }
        const float e = exp2f_fast((float)s), xp = to_f(x[k * a.xs + p]);
        float qk = 0.f;
        for (int n = part; n < N; n += parts) qk += to_f(Cm[k * a.cs + n]) * to_f(Bm[k * a.bs + n]);
        const float uk = DELTA ? to_f(beta[(int64_t)k * a.H]) * (xp - e * v - less) : xp;
        qk = sum(qk);
        if (part == 0) {
            u[k * P + p] = uk;
            y[k * ys + p] = from_f<T>(e * o + more + qk * uk + D * xp);
        }
        __syncthreads();
    }
}

template <typename T>
int run_tree(const Args& a) {
    const size_t lds = (size_t)a.T * a.P * 4;
    auto kernel = a.beta ? k_tree<T, true> : k_tree<T, false>;
    if (lds > 32 * 1024 &&
        hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
        return 7;
    kernel<<<(unsigned)(a.b * a.H), 256, lds, a.stream>>>(a);
    return hipGetLastError() == hipSuccess ? 0 : 7;
}

int tree_bf16(const Args& a);
int tree_f32(const Args& a);

}  // namespace pool
}  // namespace ssd
