// bcnorm.hpp -- the norm of every head's row of B and C (the keys and queries of the scan and
// of the delta rule), with the position rotation, in one pass over both tensors:
//
//   r = (s sum x^2 + eps)^-1/2,  s = 1/N (rms) or 1 (l2),   v = w o x r,
//   pairs (v_i, v_{i+F}), or (v_2i, v_2i+1) interleaved, turned by pos * inv_freq_i, i < F;
//   columns from 2F on pass.
//
// Backward, g the output gradient turned back: dw = sum over tokens and heads of g o x r,
// dx = r (g o w) - s r^3 x <x, g o w>.
//
// A row is VPL elements in each of N / VPL lanes; sums are butterflies among them, a pair's
// other half one shuffle away.  A work-group takes TOK tokens, so each token's cosines and
// sines (the angle and its reduction in float64: a float32 product is off by 0.06 radian at
// position 10^6) are formed once for all of its heads.  Bound by HBM: every element is read
// and written once.  8 rows of 4096 tokens, 16 heads each of 128, bfloat16: 130 us for 0.54 GB, 4.1
// TB/s; backward 176 us for 0.81 GB, 4.6 TB/s (a large copy reaches 5.1).
#pragma once

#include "device.hpp"

namespace ssd {
namespace bcnorm {

constexpr int kDwGroups = 1024;  // most work-groups of the backward (rows of its partial sums)

struct Args {
    int64_t tokens, T;  // batch * seqlen, seqlen
    int GB, GC, N, F;
    int64_t sB, sC;     // elements between tokens of B and C
    float eps;
    int l2, interleaved, tok;
    const void* B;
    const void* C;
    const float* wB;
    const float* wC;
    const float* inv_freq;
    const int* pos;     // [tokens], nullptr: the index in the row
    void* Bn;           // forward: outputs
    void* Cn;
    const void* dBn;    // backward
    const void* dCn;
    void* dB;
    void* dC;
    float* dwB;
    float* dwC;
    float* part;        // [groups][2 N]
    int groups;
    hipStream_t stream;
};

template <typename T, int VPL>
__device__ __forceinline__ void load_row(const T* p, float (&v)[VPL]) {
    if constexpr (VPL == 8) {
        const auto x = ld8(p);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = to_f(x[e]);
    } else {
        const auto x = ld4(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = to_f(x[e]);
    }
}
template <typename T, int VPL>
__device__ __forceinline__ void store_row(T* p, const float (&v)[VPL]) {
    if constexpr (VPL == 8) {
        typename V8<T>::type x;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = from_f<T>(v[e]);
        st8(p, x);
    } else {
        typename V4<T>::type x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = from_f<T>(v[e]);
        st4(p, x);
    }
}

// The cosines and sines of tokens t0 .. t0 + nt - 1 into cs[token][2][F].
__device__ __forceinline__ void angles(const Args& a, int64_t t0, int nt, float* cs) {
    for (int k = threadIdx.x; k < nt * a.F; k += 256) {
        const int tk = k / a.F, i = k - tk * a.F;
        const int64_t t = t0 + tk;
        const double p = (double)(a.pos ? a.pos[t] : (int)(t % a.T));
        const double turns = p * (double)a.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        cs[tk * 2 * a.F + i] = c;
        cs[(tk * 2 + 1) * a.F + i] = s;
    }
}

// v turned by the token's angles (sign = 1) or back (sign = -1); n0 = this lane's first column
template <int VPL>
__device__ __forceinline__ void turn(float (&v)[VPL], const float* cs, int F, int n0, bool interleaved, float sign) {
    if (interleaved) {
        if (n0 < 2 * F) {
#pragma unroll
            for (int e = 0; e < VPL; e += 2) {
                const int i = (n0 + e) >> 1;
                const float c = cs[i], s = sign * cs[F + i], p = v[e], o = v[e + 1];
                v[e] = p * c - o * s;
                v[e + 1] = p * s + o * c;
            }
        }
        return;
    }
    const bool lo = n0 < F, in = n0 < 2 * F;
    const int lane = threadIdx.x & 63, d = F / VPL;
    const int other = !in ? lane : lo ? lane + d : lane - d;
#pragma unroll
    for (int e = 0; e < VPL; ++e) {
        const float o = __shfl(v[e], other, 64);
        if (in) {
            const int i = (lo ? n0 : n0 - F) + e;
            v[e] = v[e] * cs[i] + (lo ? -o : o) * (sign * cs[F + i]);
        }
    }
}

__device__ __forceinline__ float row_sum(float s, int R) {
    for (int off = R >> 1; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
    return s;
}

// 1 / sqrt(scale |v|^2 + eps) of a row, v left as it is and k = 1; a row whose squares' sum leaves
// float32 (values of 10^18 and more) is scaled by k = 2^-70 first, far past eps.
template <int VPL>
__device__ __forceinline__ float row_root(float (&v)[VPL], int R, float scale, float eps, float& k) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < VPL; ++e) s += v[e] * v[e];
    s = row_sum(s, R);
    float r = 1.f / sqrtf(s * scale + eps);
    const bool over = s > 3.4028235e38f;
    k = 1.f;
    if (__any(over)) {
        k = over ? 0x1p-70f : 1.f;
        s = 0.f;
#pragma unroll
        for (int e = 0; e < VPL; ++e) {
            v[e] *= k;
            s += v[e] * v[e];
        }
        s = row_sum(s, R);
        if (over) r = 1.f / sqrtf(s * scale);
    }
    return r;
}

template <typename T, int VPL>
__global__ __launch_bounds__(256) void k_bc_norm(Args a) {
    extern __shared__ float cs[];
    const int R = a.N / VPL, rows = 256 / R, heads = a.GB + a.GC;
    const int rg = threadIdx.x / R, n0 = (threadIdx.x % R) * VPL;
    const int64_t t0 = (int64_t)blockIdx.x * a.tok;
    const int nt = (int)min((int64_t)a.tok, a.tokens - t0);
    if (a.F) {
        angles(a, t0, nt, cs);
        __syncthreads();
    }
    const float scale = a.l2 ? 1.f : 1.f / (float)a.N;
    float wb[VPL], wc[VPL];
#pragma unroll
    for (int e = 0; e < VPL; ++e) {
        wb[e] = a.wB ? a.wB[n0 + e] : 1.f;
        wc[e] = a.wC ? a.wC[n0 + e] : 1.f;
    }
    for (int base = 0; base < nt * heads; base += rows) {
        const int it = base + rg;
        const bool on = it < nt * heads;  // idle lanes still take part in the shuffles
        const int tk = on ? it / heads : 0, hd = on ? it - tk * heads : 0;
        const int64_t t = t0 + tk;
        const bool isB = hd < a.GB;
        const T* src = isB ? static_cast<const T*>(a.B) + t * a.sB + hd * a.N
                           : static_cast<const T*>(a.C) + t * a.sC + (hd - a.GB) * a.N;
        float v[VPL], k;
        load_row<T, VPL>(src + n0, v);
        const float r = row_root<VPL>(v, R, scale, a.eps, k);
#pragma unroll
        for (int e = 0; e < VPL; ++e) v[e] = v[e] * r * (isB ? wb[e] : wc[e]);
        if (a.F) turn<VPL>(v, cs + tk * 2 * a.F, a.F, n0, a.interleaved, 1.f);
        T* dst = isB ? static_cast<T*>(a.Bn) + (t * a.GB + hd) * a.N
                     : static_cast<T*>(a.Cn) + (t * a.GC + hd - a.GB) * a.N;
        if (on) store_row<T, VPL>(dst + n0, v);
    }
}

template <typename T, int VPL>
__global__ __launch_bounds__(256) void k_bc_norm_bwd(Args a) {
    extern __shared__ float cs[];  // angles, then the weights' sums [256 / R][N] twice
    const int R = a.N / VPL, rows = 256 / R, heads = a.GB + a.GC;
    const int rg = threadIdx.x / R, n0 = (threadIdx.x % R) * VPL;
    const float scale = a.l2 ? 1.f : 1.f / (float)a.N;
    float wb[VPL], wc[VPL], gb[VPL], gc[VPL];
#pragma unroll
    for (int e = 0; e < VPL; ++e) {
        wb[e] = a.wB ? a.wB[n0 + e] : 1.f;
        wc[e] = a.wC ? a.wC[n0 + e] : 1.f;
        gb[e] = gc[e] = 0.f;
    }
    for (int64_t t0 = (int64_t)blockIdx.x * a.tok; t0 < a.tokens; t0 += (int64_t)a.groups * a.tok) {
        const int nt = (int)min((int64_t)a.tok, a.tokens - t0);
        if (a.F) {
            __syncthreads();
            angles(a, t0, nt, cs);
            __syncthreads();
        }
        for (int base = 0; base < nt * heads; base += rows) {
            const int it = base + rg;
            const bool on = it < nt * heads;
            const int tk = on ? it / heads : 0, hd = on ? it - tk * heads : 0;
            const int64_t t = t0 + tk;
            const bool isB = hd < a.GB;
            const int64_t o = isB ? (t * a.GB + hd) * a.N : (t * a.GC + hd - a.GB) * a.N;
            const T* src = isB ? static_cast<const T*>(a.B) + t * a.sB + hd * a.N
                               : static_cast<const T*>(a.C) + t * a.sC + (hd - a.GB) * a.N;
            float x[VPL], g[VPL];
            load_row<T, VPL>(src + n0, x);
            load_row<T, VPL>(static_cast<const T*>(isB ? a.dBn : a.dCn) + o + n0, g);
            if (a.F) turn<VPL>(g, cs + tk * 2 * a.F, a.F, n0, a.interleaved, -1.f);
            float d = 0.f, k;
            const float r = row_root<VPL>(x, R, scale, a.eps, k);
#pragma unroll
            for (int e = 0; e < VPL; ++e) {
                const float xr = x[e] * r;
                if (on) {
                    if (isB) gb[e] += g[e] * xr;
                    else gc[e] += g[e] * xr;
                }
                g[e] *= isB ? wb[e] : wc[e];
                x[e] = xr;
                d += xr * g[e];
            }
            d = row_sum(d, R) * scale;
#pragma unroll
            for (int e = 0; e < VPL; ++e) g[e] = r * k * (g[e] - x[e] * d);
            if (on) store_row<T, VPL>(static_cast<T*>(isB ? a.dB : a.dC) + o + n0, g);
        }
    }
    if (!a.part) return;
    // this work-group's sums over its rows, in row-group order
    __syncthreads();
    float* red = cs;  // [2][rows][N]
#pragma unroll
    for (int e = 0; e < VPL; ++e) {
        red[rg * a.N + n0 + e] = gb[e];
        red[(rows + rg) * a.N + n0 + e] = gc[e];
    }
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * a.N; k += 256) {
        const int side = k / a.N, n = k - side * a.N;
        float s = 0.f;
        for (int j = 0; j < rows; ++j) s += red[(side * rows + j) * a.N + n];
        a.part[(int64_t)blockIdx.x * 2 * a.N + k] = s;
    }
}

// dwB and dwC from the work-groups' sums, in a fixed order, in float64: 4 columns per
// work-group, 64 runs of every 64th row (with 32 columns of 8 runs, few work-groups of long
// dependent sums, it took 40 us at 1024 rows of 256)
template <int BLOCK = 256>
__global__ __launch_bounds__(BLOCK) void k_bc_norm_dw(const float* __restrict__ part, float* __restrict__ dwB,
                                                      float* __restrict__ dwC, int N, int groups) {
    constexpr int RUNS = BLOCK / 4;
    __shared__ double red[BLOCK];
    const int k = blockIdx.x * 4 + (threadIdx.x & 3), j = threadIdx.x >> 2;
    double s = 0.0;
#pragma unroll 4
    for (int gr = j; gr < groups; gr += RUNS) s += (double)part[(int64_t)gr * 2 * N + k];
    red[threadIdx.x] = s;
    __syncthreads();
    for (int half = RUNS / 2; half > 0; half >>= 1) {
        if (j < half) red[threadIdx.x] += red[threadIdx.x + 4 * half];
        __syncthreads();
    }
    if (j == 0) {
        s = red[threadIdx.x];
        if (k < N) {
            if (dwB) dwB[k] = (float)s;
        } else if (dwC) {
            dwC[k - N] = (float)s;
        }
    }
}

// Elements per lane: 8 (16-byte bfloat16 accesses), or 4 where 8 would straddle the halves of
// the rotation.
inline int per_lane(const Args& a) { return a.F % 8 && !a.interleaved ? 4 : 8; }

template <typename T, int VPL>
int launch(const Args& a, bool bwd) {
    const size_t ang = (size_t)a.tok * 2 * a.F * 4;
    if (!bwd) {
        k_bc_norm<T, VPL><<<(unsigned)((a.tokens + a.tok - 1) / a.tok), 256, ang, a.stream>>>(a);
    } else {
        const size_t red = a.part ? (size_t)2 * 256 * VPL * 4 : 0;
        k_bc_norm_bwd<T, VPL><<<(unsigned)a.groups, 256, ang > red ? ang : red, a.stream>>>(a);
        if (a.part) k_bc_norm_dw<256><<<(unsigned)(2 * a.N / 4), 256, 0, a.stream>>>(a.part, a.dwB, a.dwC, a.N, a.groups);
    }
    return hipGetLastError() == hipSuccess ? 0 : 7;
}
template <typename T>
int run(const Args& a, bool bwd) {
    return per_lane(a) == 8 ? launch<T, 8>(a, bwd) : launch<T, 4>(a, bwd);
}

}  // namespace bcnorm
}  // namespace ssd
