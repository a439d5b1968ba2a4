// delta_abi.hip -- the C ABI of the gated delta rule and of the norm of B and C (declared in
// include/ssd.h): host-side validation, workspace layout, launches.  No allocation, no
// global state; every check happens before the first HIP call.
#include <math.h>
#include <string.h>

#include "abi_common.hpp"
#include "bcnorm.hpp"
#include "delta_launch.hpp"

namespace {

using ssd::delta::kTab;
using ssd::delta::kVec;

constexpr int64_t kReach = 0x7fff0000;  // bytes that a kernel addresses from one base

int check_delta(const ssd_problem* p, bool packed) {
    const int st = check_problem(p);
    if (st) return st;
    if (p->chunk != ssd::delta::L || p->flags != 0) return SSD_ERR_UNSUPPORTED;
    const int64_t b = p->batch, T = p->seqlen, H = p->nheads;
    const int64_t nc = (T + p->chunk - 1) / p->chunk;
    const int64_t tabs = packed ? nc + b : b * nc;
    // one work-group per (chunk, head), and per (row, head, 16 columns)
    if (!grid_ok(tabs * H, 256) || !grid_ok(b * H * (p->headdim / 16), 512)) return SSD_ERR_UNSUPPORTED;
    // a chunk's rows lie within 2 GiB (B's and C's do: check_problem bounds the groups)
    if (H * p->headdim * (int64_t)esize(p->dtype) * p->chunk > kReach) return SSD_ERR_UNSUPPORTED;
    if (packed && T > 0x7fffffffLL) return SSD_ERR_UNSUPPORTED;  // int32 offsets
    return SSD_OK;
}

// Workspace: S, M and the decay factors of every (chunk, head); the packed row map; for the
// backward also the residuals, the adjoint's z, e^c K h^T, the entering states and adjoints of
// every chunk and the partial sums.
struct Layout {
    size_t tab, vec, ts, kb, order, r, rlo, rll, z, zlo, zll, kh, hin, hlo, lin, fq, fk, dj, tot, dAp, part, total;
    int64_t ntab, slices, tots, nsub;
};

Layout layout_of(const ssd_problem* p, bool packed, bool bwd) {
    Layout o;
    memset(&o, 0, sizeof(o));
    const int64_t b = p->batch, T = p->seqlen, H = p->nheads, P = p->headdim, N = p->dstate, G = p->ngroups;
    const int64_t nc = (T + ssd::delta::L - 1) / ssd::delta::L;
    const size_t es = esize(p->dtype);
    o.ntab = packed ? nc + b : b * nc;
    size_t off = 0;
    auto take = [&](size_t& at, size_t bytes) {
        at = off;
        off += align_up(bytes);
    };
    const bool frag = ssd::delta::dma_walk(p->dtype == SSD_BF16, N);
    take(o.tab, (size_t)(o.ntab * H) * (!frag ? kTab * 4
                                        : ((bwd ? ssd::delta::kFragTab2 : ssd::delta::kFragTab) + ssd::delta::kFragVec) * 2));
    if (bwd || !frag) take(o.vec, (size_t)(o.ntab * H) * kVec * 4);
    if (packed) {
        take(o.ts, (size_t)(b + 1) * 4);
        take(o.kb, (size_t)(b + 1) * 4);
        take(o.order, (size_t)b * 4);
    }
    if (bwd) {
        o.slices = ssd::delta::bwd_slices(p->dtype == SSD_BF16, b * H, P, N);
        o.tots = ssd::delta::bwd_tots(p->dtype == SSD_BF16, b * H, P, N);
        o.nsub = ssd::delta::grad_shares(o.ntab, H, G, N);
        take(o.r, (size_t)(b * T * H * P) * es);
        take(o.z, (size_t)(b * T * H * P) * es);
        if (es == 2)
            for (size_t* at : {&o.rlo, &o.zlo, &o.rll, &o.zll}) take(*at, (size_t)(b * T * H * P) * es);
        take(o.kh, (size_t)(o.ntab * H * ssd::delta::L * P) * 4);
        take(o.hin, (size_t)(o.ntab * H * P * N) * es);
        if (es == 2) take(o.hlo, (size_t)(o.ntab * H * P * N) * 2);
        take(o.lin, (size_t)(o.ntab * H * P * N) * es);
        for (size_t* at : {&o.fq, &o.fk, &o.dj}) take(*at, (size_t)(o.slices * b * H * T) * 4);
        take(o.tot, (size_t)(o.tots * o.ntab * H) * 4);
        take(o.dAp, (size_t)(o.ntab * H) * 8);
        if (o.nsub > 1) take(o.part, (size_t)(o.nsub * 2 * b * T * G * N) * 4);
    }
    o.total = (b == 0 || T == 0) ? 0 : off;
    return o;
}

ssd::delta::Args args_of(const ssd_problem* p, const Layout& o, void* ws, void* stream, bool packed) {
    ssd::delta::Args a;
    memset(&a, 0, sizeof(a));
    char* w = static_cast<char*>(ws);
    a.T = p->seqlen;
    a.H = (int)p->nheads;
    a.P = (int)p->headdim;
    a.N = (int)p->dstate;
    a.G = (int)p->ngroups;
    a.nc = (int)((p->seqlen + ssd::delta::L - 1) / ssd::delta::L);
    a.ntab = (int)o.ntab;
    a.rows.ts = packed ? reinterpret_cast<int*>(w + o.ts) : nullptr;
    a.rows.kb = packed ? reinterpret_cast<int*>(w + o.kb) : nullptr;
    a.order = packed ? reinterpret_cast<int*>(w + o.order) : nullptr;
    a.rows.T = a.T;
    a.rows.nc = a.nc;
    a.rows.nrows = (int)p->batch;
    a.rows.H = a.H;
    a.rows.kcap = a.ntab;
    a.tab = reinterpret_cast<float*>(w + o.tab);
    a.vec = reinterpret_cast<float*>(w + o.vec);
    a.stream = (hipStream_t)stream;
    return a;
}

bool any_overlap(const Range* outs, int no, const Range* ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

int delta_fwd(const ssd_problem* p, const int32_t* cu, bool packed, const void* x, const float* dt, const float* A,
              const void* B, const void* C, const void* beta, const float* h0, void* y, float* hT, void* ws,
              size_t ws_bytes, void* stream) {
    const int st = check_delta(p, packed);
    if (st) return st;
    const int64_t b = p->batch, T = p->seqlen, H = p->nheads, P = p->headdim, N = p->dstate, G = p->ngroups;
    const size_t es = esize(p->dtype), state = (size_t)(b * H * P * N) * 4;
    const int64_t tok = packed ? T : b * T;
    if (b == 0) return SSD_OK;
    if (!A) return SSD_ERR_NULL;
    if (!aligned(A, 4) || (h0 && !aligned(h0, 16)) || (hT && !aligned(hT, 16))) return SSD_ERR_ALIGN;
    if (T == 0) {
        if (!hT) return SSD_OK;
        if (overlap({hT, state}, {h0, state})) return SSD_ERR_ALIAS;
        return copy_state(h0, hT, b * H * P * N, stream);
    }
    if (!x || !dt || !B || !C || !beta || !y || (packed && !cu)) return SSD_ERR_NULL;
    if (!aligned(x, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(y, 16) || !aligned(dt, 4) ||
        !aligned(beta, es) || (packed && !aligned(cu, 4)))
        return SSD_ERR_ALIGN;
    const Layout o = layout_of(p, packed, false);
    if (!ws || ws_bytes < o.total) return SSD_ERR_WORKSPACE;
    if (!aligned(ws, kAlign)) return SSD_ERR_ALIGN;
    const Range rws = {ws, o.total}, rcu = {cu, packed ? (size_t)(b + 1) * 4 : 0};
    const Range ins[] = {{x, (size_t)(tok * H * P) * es}, {dt, (size_t)(tok * H) * 4}, {A, (size_t)H * 4},
                         {B, (size_t)(tok * G * N) * es}, {C, (size_t)(tok * G * N) * es},
                         {beta, (size_t)(tok * H) * es},  {h0, h0 ? state : 0},         rcu, rws};
    const Range outs[] = {{y, (size_t)(tok * H * P) * es}, {hT, hT ? state : 0}};
    if (any_overlap(outs, 2, ins, 9) || overlap(rcu, rws)) return SSD_ERR_ALIAS;

    ssd::delta::Args a = args_of(p, o, ws, stream, packed);
    a.x = x; a.dt = dt; a.A = A; a.B = B; a.C = C; a.beta = beta; a.h0 = h0; a.y = y; a.hT = hT;
    if (packed) {
        ssd::k_rows<1024><<<1, 1024, 0, a.stream>>>(cu, (int)b, T, ssd::delta::L, const_cast<int*>(a.rows.ts),
                                                    const_cast<int*>(a.rows.kb));
        if (hipGetLastError() != hipSuccess) return SSD_ERR_HIP;
    }
    return p->dtype == SSD_BF16 ? ssd::delta::run_bf16(a, false) : ssd::delta::run_f32(a, false);
}

int check_delta_bwd(const ssd_problem* p) {
    const int st = check_delta(p, false);
    if (st) return st;
    const int64_t b = p->batch, T = p->seqlen, H = p->nheads, G = p->ngroups, N = p->dstate;
    const int64_t nc = (T + p->chunk - 1) / p->chunk;
    const int64_t nsub = ssd::delta::grad_shares(b * nc, H, G, N);
    if (!grid_ok(b * nc * G * nsub * (N > 64 ? N / 64 : 1), 256) || !grid_ok(2 * b * T * G * N / 4 / 256 + 1, 256))
        return SSD_ERR_UNSUPPORTED;
    // the states of a chunk's heads lie within 2 GiB
    if (H * p->headdim * N * (int64_t)esize(p->dtype) > kReach) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

int delta_bwd(const ssd_problem* p, const void* x, const float* dt, const float* A, const void* B, const void* C,
              const void* beta, const float* h0, const void* dy, const float* dhT, void* dx, float* ddt, float* dA,
              void* dB, void* dC, void* dbeta, float* dh0, void* ws, size_t ws_bytes, void* stream) {
    const int st = check_delta_bwd(p);
    if (st) return st;
    const int64_t b = p->batch, T = p->seqlen, H = p->nheads, P = p->headdim, N = p->dstate, G = p->ngroups;
    const size_t es = esize(p->dtype), state = (size_t)(b * H * P * N) * 4, ab = (size_t)H * 4;
    if (!A || !dA) return SSD_ERR_NULL;
    if (!aligned(A, 4) || !aligned(dA, 4) || (h0 && !aligned(h0, 16)) || (dhT && !aligned(dhT, 16)) ||
        (dh0 && !aligned(dh0, 16)))
        return SSD_ERR_ALIGN;
    const Range rA = {A, ab}, rh0 = {h0, h0 ? state : 0}, rdhT = {dhT, dhT ? state : 0};
    const Range rdA = {dA, ab}, rdh0 = {dh0, dh0 ? state : 0};
    if (b == 0 || T == 0) {  // no tokens: dA = 0, dh0 = dhT
        const Range in[] = {rA, rh0, rdhT}, out[] = {rdA, rdh0};
        if (any_overlap(out, 2, in, 3)) return SSD_ERR_ALIAS;
        k_zero<<<(unsigned)((H + 255) / 256), 256, 0, (hipStream_t)stream>>>(dA, H);
        if (dh0 && b > 0) return copy_state(dhT, dh0, b * H * P * N, stream);
        return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
    }
    if (!x || !dt || !B || !C || !beta || !dy || !dx || !ddt || !dB || !dC || !dbeta) return SSD_ERR_NULL;
    const void* a16[] = {x, B, C, dy, dx, dB, dC};
    for (const void* v : a16)
        if (!aligned(v, 16)) return SSD_ERR_ALIGN;
    if (!aligned(dt, 4) || !aligned(ddt, 4) || !aligned(beta, es) || !aligned(dbeta, es)) return SSD_ERR_ALIGN;
    const Layout o = layout_of(p, false, true);
    if (!ws || ws_bytes < o.total) return SSD_ERR_WORKSPACE;
    if (!aligned(ws, kAlign)) return SSD_ERR_ALIGN;
    const size_t xb = (size_t)(b * T * H * P) * es, bc = (size_t)(b * T * G * N) * es, gt = (size_t)(b * T * H);
    const Range ins[] = {{x, xb}, {dt, gt * 4}, rA, {B, bc}, {C, bc}, {beta, gt * es}, rh0, {dy, xb}, rdhT,
                         {ws, o.total}};
    const Range outs[] = {{dx, xb}, {ddt, gt * 4}, rdA, {dB, bc}, {dC, bc}, {dbeta, gt * es}, rdh0};
    if (any_overlap(outs, 7, ins, 10)) return SSD_ERR_ALIAS;

    ssd::delta::Args a = args_of(p, o, ws, stream, false);
    char* w = static_cast<char*>(ws);
    a.x = x; a.dt = dt; a.A = A; a.B = B; a.C = C; a.beta = beta; a.h0 = h0; a.dy = dy; a.dhT = dhT;
    a.dx = dx; a.ddt = ddt; a.dA = dA; a.dB = dB; a.dC = dC; a.dbeta = dbeta; a.dh0 = dh0;
    a.r = w + o.r;
    a.rlo = w + o.rlo;
    a.rll = w + o.rll;
    a.z = w + o.z;
    a.zlo = w + o.zlo;
    a.zll = w + o.zll;
    a.kh = reinterpret_cast<float*>(w + o.kh);
    a.hin = w + o.hin;
    a.lin = w + o.lin;
    a.hlo = reinterpret_cast<short*>(w + o.hlo);
    a.fq = reinterpret_cast<float*>(w + o.fq);
    a.fk = reinterpret_cast<float*>(w + o.fk);
    a.dj = reinterpret_cast<float*>(w + o.dj);
    a.tot = reinterpret_cast<float*>(w + o.tot);
    a.dAp = reinterpret_cast<double*>(w + o.dAp);
    a.part = o.nsub > 1 ? reinterpret_cast<float*>(w + o.part) : nullptr;
    a.slices = (int)o.slices;
    a.tots = (int)o.tots;
    a.nsub = (int)o.nsub;
    return p->dtype == SSD_BF16 ? ssd::delta::run_bf16(a, true) : ssd::delta::run_f32(a, true);
}

int delta_step(const ssd_problem* p, const void* x, const float* dt, const float* A, const void* B, const void* C,
               const void* beta, float* h, void* y, void* stream) {
    if (!p) return SSD_ERR_NULL;
    if (p->batch < 0 || p->seqlen < 0 || p->nheads <= 0 || p->headdim <= 0 || p->dstate <= 0 || p->ngroups <= 0 ||
        p->nheads % p->ngroups != 0)
        return SSD_ERR_SHAPE;
    if (p->dtype != SSD_F32 && p->dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (!pn_supported(p->headdim, p->dstate) || p->flags != 0) return SSD_ERR_UNSUPPORTED;
    const int64_t b = p->batch, T = p->seqlen, H = p->nheads, P = p->headdim, N = p->dstate, G = p->ngroups;
    if (H > (int64_t)1 << 20 || b > 0x7fffffffLL || !grid_ok(b * H, 256) || T > (int64_t)1 << 32 ||
        b * T > ((int64_t)1 << 40) / (H * (P > N ? P : N)))
        return SSD_ERR_UNSUPPORTED;
    if (b == 0 || T == 0) return SSD_OK;  // h is left as it is
    if (!x || !dt || !A || !B || !C || !beta || !h || !y) return SSD_ERR_NULL;
    const size_t es = esize(p->dtype);
    if (!aligned(h, 16) || !aligned(dt, 4) || !aligned(A, 4) || !aligned(x, es) || !aligned(y, es) ||
        !aligned(beta, es) || !aligned(B, 16) || !aligned(C, 16))
        return SSD_ERR_ALIGN;
    const size_t xb = (size_t)(b * T * H * P) * es, bc = (size_t)(b * T * G * N) * es;
    const Range ins[] = {{x, xb}, {dt, (size_t)(b * T * H) * 4}, {A, (size_t)H * 4}, {B, bc}, {C, bc},
                         {beta, (size_t)(b * T * H) * es}};
    const Range outs[] = {{h, (size_t)(b * H * P * N) * 4}, {y, xb}};
    if (any_overlap(outs, 2, ins, 6)) return SSD_ERR_ALIAS;
    const dim3 grid((unsigned)(b * H), (unsigned)((P * N + 2047) / 2048));
    hipStream_t s = (hipStream_t)stream;
    if (p->dtype == SSD_BF16) {
        typedef ssd::bf16 E;
        ssd::delta::k_delta_step<E><<<grid, 256, 0, s>>>(
            static_cast<const E*>(x), dt, A, static_cast<const E*>(B), static_cast<const E*>(C),
            static_cast<const E*>(beta), h, static_cast<E*>(y), T, (int)H, (int)P, (int)N, (int)G);
    } else {
        ssd::delta::k_delta_step<float><<<grid, 256, 0, s>>>(
            static_cast<const float*>(x), dt, A, static_cast<const float*>(B), static_cast<const float*>(C),
            static_cast<const float*>(beta), h, static_cast<float*>(y), T, (int)H, (int)P, (int)N, (int)G);
    }
    return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

// ---- the norm of B and C ----
int check_norm(const ssd_norm* p) {
    if (!p) return SSD_ERR_NULL;
    if (p->batch < 0 || p->seqlen < 0 || p->bheads < 0 || p->cheads < 0 || p->bheads + p->cheads <= 0 ||
        p->dstate <= 0 || p->pairs < 0 || 2 * p->pairs > p->dstate)
        return SSD_ERR_SHAPE;
    if (p->dtype != SSD_F32 && p->dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (!pn_supported(16, p->dstate) || p->pairs % 4 != 0) return SSD_ERR_UNSUPPORTED;
    if ((p->mode != SSD_NORM_RMS && p->mode != SSD_NORM_L2) || (p->interleaved != 0 && p->interleaved != 1))
        return SSD_ERR_UNSUPPORTED;
    if (!(p->eps > 0.f) || isinf(p->eps)) return SSD_ERR_UNSUPPORTED;
    if (p->bheads > 1 << 16 || p->cheads > 1 << 16 || p->batch > (int64_t)1 << 31 || p->seqlen > (int64_t)1 << 31)
        return SSD_ERR_UNSUPPORTED;
    if (p->batch * p->seqlen > kMaxThreads / 256) return SSD_ERR_UNSUPPORTED;
    if (p->batch > 0 && p->seqlen > 0) {
        if (p->bstride < p->bheads * p->dstate || p->cstride < p->cheads * p->dstate) return SSD_ERR_SHAPE;
        if (p->bstride > (int64_t)1 << 32 || p->cstride > (int64_t)1 << 32) return SSD_ERR_UNSUPPORTED;
    }
    return SSD_OK;
}

ssd::bcnorm::Args norm_args(const ssd_norm* p, void* stream) {
    ssd::bcnorm::Args a;
    memset(&a, 0, sizeof(a));
    a.tokens = p->batch * p->seqlen;
    a.T = p->seqlen;
    a.GB = (int)p->bheads;
    a.GC = (int)p->cheads;
    a.N = (int)p->dstate;
    a.F = (int)p->pairs;
    a.sB = p->bstride;
    a.sC = p->cstride;
    a.eps = p->eps;
    a.l2 = p->mode == SSD_NORM_L2;
    a.interleaved = p->interleaved;
    // tokens per work-group: one while that already fills the GPU with work-groups or less; from 2048
    // tokens four, so that a token's angles and a work-group's start cost less (one / four, us, 16 + 16
    // heads of 128: 512 tokens 8.6 / 13.9, 2048 tokens 21.9 / 17.8, backward 27.8 / 26.6, 32768 tokens 253 / 149,
    // 208 / 199; 1 + 1 heads: 512 tokens 7.1 / 5.3, 2048 tokens 18.3 / 7.2, 21.4 / 12.7)
    a.tok = a.tokens >= 2048 ? 4 : 1;
    a.groups = (int)((a.tokens + a.tok - 1) / a.tok);
    if (a.groups > ssd::bcnorm::kDwGroups) a.groups = ssd::bcnorm::kDwGroups;
    a.stream = (hipStream_t)stream;
    return a;
}

// bytes from a strided tensor's first element to its last
size_t span(int64_t tokens, int64_t stride, int64_t heads, int64_t N, size_t es) {
    return heads ? (size_t)((tokens - 1) * stride + heads * N) * es : 0;
}

int norm_common(const ssd_norm* p, const void* B, const void* C, const float* wB, const float* wC,
                const float* inv_freq, const int32_t* pos) {
    const size_t es = esize(p->dtype);
    if ((p->bheads && !B) || (p->cheads && !C) || (p->pairs && !inv_freq)) return SSD_ERR_NULL;
    if (!aligned(B, 16) || !aligned(C, 16) || (p->bheads && p->bstride * es % 16) ||
        (p->cheads && p->cstride * es % 16) || !aligned(wB, 4) || !aligned(wC, 4) || !aligned(inv_freq, 4) ||
        !aligned(pos, 4))
        return SSD_ERR_ALIGN;
    return SSD_OK;
}

int bc_norm(const ssd_norm* p, const void* B, const void* C, const float* wB, const float* wC,
            const float* inv_freq, const int32_t* pos, void* Bn, void* Cn, void* stream) {
    int st = check_norm(p);
    if (st) return st;
    const int64_t tok = p->batch * p->seqlen;
    if (tok == 0) return SSD_OK;
    st = norm_common(p, B, C, wB, wC, inv_freq, pos);
    if (st) return st;
    if ((p->bheads && !Bn) || (p->cheads && !Cn)) return SSD_ERR_NULL;
    if (!aligned(Bn, 16) || !aligned(Cn, 16)) return SSD_ERR_ALIGN;
    const size_t es = esize(p->dtype), w = (size_t)p->dstate * 4;
    const Range ins[] = {{B, span(tok, p->bstride, p->bheads, p->dstate, es)},
                         {C, span(tok, p->cstride, p->cheads, p->dstate, es)},
                         {wB, w}, {wC, w}, {inv_freq, (size_t)p->pairs * 4}, {pos, (size_t)tok * 4}};
    const Range outs[] = {{Bn, (size_t)(tok * p->bheads * p->dstate) * es},
                          {Cn, (size_t)(tok * p->cheads * p->dstate) * es}};
    if (any_overlap(outs, 2, ins, 6)) return SSD_ERR_ALIAS;
    ssd::bcnorm::Args a = norm_args(p, stream);
    a.B = B; a.C = C; a.wB = wB; a.wC = wC; a.inv_freq = inv_freq; a.pos = pos; a.Bn = Bn; a.Cn = Cn;
    return p->dtype == SSD_BF16 ? ssd::bcnorm::run<ssd::bf16>(a, false) : ssd::bcnorm::run<float>(a, false);
}

int bc_norm_bwd(const ssd_norm* p, const void* B, const void* C, const float* wB, const float* wC,
                const float* inv_freq, const int32_t* pos, const void* dBn, const void* dCn, void* dB, void* dC,
                float* dwB, float* dwC, void* ws, size_t ws_bytes, void* stream) {
    int st = check_norm(p);
    if (st) return st;
    const int64_t tok = p->batch * p->seqlen;
    const size_t es = esize(p->dtype), w = (size_t)p->dstate * 4;
    if (!aligned(dwB, 4) || !aligned(dwC, 4)) return SSD_ERR_ALIGN;
    const Range rwB = {dwB, w}, rwC = {dwC, w};
    if (tok == 0) {  // no tokens: the weights' gradients are zero
        if (overlap(rwB, rwC) || overlap(rwB, {wB, w}) || overlap(rwB, {wC, w}) || overlap(rwC, {wB, w}) ||
            overlap(rwC, {wC, w}))
            return SSD_ERR_ALIAS;
        for (float* d : {dwB, dwC})
            if (d) k_zero<<<1, 256, 0, (hipStream_t)stream>>>(d, p->dstate);
        return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
    }
    st = norm_common(p, B, C, wB, wC, inv_freq, pos);
    if (st) return st;
    if ((p->bheads && (!dBn || !dB)) || (p->cheads && (!dCn || !dC))) return SSD_ERR_NULL;
    if (!aligned(dBn, 16) || !aligned(dCn, 16) || !aligned(dB, 16) || !aligned(dC, 16)) return SSD_ERR_ALIGN;
    ssd::bcnorm::Args a = norm_args(p, stream);
    const size_t need = dwB || dwC ? align_up((size_t)a.groups * 2 * w) : 0;
    if (need && (!ws || ws_bytes < need)) return SSD_ERR_WORKSPACE;
    if (need && !aligned(ws, kAlign)) return SSD_ERR_ALIGN;
    const size_t nb = (size_t)(tok * p->bheads * p->dstate) * es, ncb = (size_t)(tok * p->cheads * p->dstate) * es;
    const Range ins[] = {{B, span(tok, p->bstride, p->bheads, p->dstate, es)},
                         {C, span(tok, p->cstride, p->cheads, p->dstate, es)},
                         {wB, w}, {wC, w}, {inv_freq, (size_t)p->pairs * 4}, {pos, (size_t)tok * 4},
                         {dBn, nb}, {dCn, ncb}, {ws, need}};
    const Range outs[] = {{dB, nb}, {dC, ncb}, rwB, rwC};
    if (any_overlap(outs, 4, ins, 9)) return SSD_ERR_ALIAS;
    a.B = B; a.C = C; a.wB = wB; a.wC = wC; a.inv_freq = inv_freq; a.pos = pos;
    a.dBn = dBn; a.dCn = dCn; a.dB = dB; a.dC = dC; a.dwB = dwB; a.dwC = dwC;
    a.part = need ? static_cast<float*>(ws) : nullptr;
    return p->dtype == SSD_BF16 ? ssd::bcnorm::run<ssd::bf16>(a, true) : ssd::bcnorm::run<float>(a, true);
}

}  // namespace

extern "C" {

size_t ssd_delta_workspace_bytes(const ssd_problem* p) {
    return check_delta(p, false) ? 0 : layout_of(p, false, false).total;
}
int ssd_delta_fwd(const ssd_problem* p, const void* x, const float* dt, const float* A, const void* B, const void* C,
                  const void* beta, const float* h0, void* y, float* hT, void* ws, size_t ws_bytes, void* stream) {
    return delta_fwd(p, nullptr, false, x, dt, A, B, C, beta, h0, y, hT, ws, ws_bytes, stream);
}

size_t ssd_delta_varlen_workspace_bytes(const ssd_problem* p) {
    return check_delta(p, true) ? 0 : layout_of(p, true, false).total;
}
int ssd_delta_fwd_varlen(const ssd_problem* p, const int32_t* cu_seqlens, const void* x, const float* dt,
                         const float* A, const void* B, const void* C, const void* beta, const float* h0, void* y,
                         float* hT, void* ws, size_t ws_bytes, void* stream) {
    return delta_fwd(p, cu_seqlens, true, x, dt, A, B, C, beta, h0, y, hT, ws, ws_bytes, stream);
}

int ssd_delta_step(const ssd_problem* p, const void* x, const float* dt, const float* A, const void* B, const void* C,
                   const void* beta, float* h, void* y, void* stream) {
    return delta_step(p, x, dt, A, B, C, beta, h, y, stream);
}

size_t ssd_delta_bwd_workspace_bytes(const ssd_problem* p) {
    return check_delta_bwd(p) ? 0 : layout_of(p, false, true).total;
}
int ssd_delta_bwd(const ssd_problem* p, const void* x, const float* dt, const float* A, const void* B, const void* C,
                  const void* beta, const float* h0, const void* dy, const float* dhT, void* dx, float* ddt, float* dA,
                  void* dB, void* dC, void* dbeta, float* dh0, void* ws, size_t ws_bytes, void* stream) {
    return delta_bwd(p, x, dt, A, B, C, beta, h0, dy, dhT, dx, ddt, dA, dB, dC, dbeta, dh0, ws, ws_bytes, stream);
}

int ssd_bc_norm(const ssd_norm* p, const void* B, const void* C, const float* wB, const float* wC,
                const float* inv_freq, const int32_t* positions, void* Bn, void* Cn, void* stream) {
    return bc_norm(p, B, C, wB, wC, inv_freq, positions, Bn, Cn, stream);
}
size_t ssd_bc_norm_bwd_workspace_bytes(const ssd_norm* p) {
    if (check_norm(p) || p->batch * p->seqlen == 0) return 0;
    return align_up((size_t)norm_args(p, nullptr).groups * 2 * (size_t)p->dstate * 4);
}
int ssd_bc_norm_bwd(const ssd_norm* p, const void* B, const void* C, const float* wB, const float* wC,
                    const float* inv_freq, const int32_t* positions, const void* dBn, const void* dCn, void* dB,
                    void* dC, float* dwB, float* dwC, void* ws, size_t ws_bytes, void* stream) {
    return bc_norm_bwd(p, B, C, wB, wC, inv_freq, positions, dBn, dCn, dB, dC, dwB, dwC, ws, ws_bytes, stream);
}

}  // extern "C"
