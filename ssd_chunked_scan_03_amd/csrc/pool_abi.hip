// pool_abi.hip -- the C ABI of the states in a pool (declared in include/ssd.h): host-side validation
// and launches.  No allocation, no global state; every check happens before the first HIP call.
#include <string.h>

#include "abi_common.hpp"
#include "pages.hpp"
#include "pool.hpp"

namespace ssd {
namespace pool {
int tree_bf16(const Args& a);
int tree_f32(const Args& a);
}  // namespace pool
}  // namespace ssd

namespace {

using ssd::pool::Args;

bool any_overlap(const Range* outs, int no, const Range* ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

constexpr int64_t kFar = (int64_t)1 << 40;  // elements that a tensor spans at most

// The pool call's operands; which of them a call has is its own matter.
struct Call {
    const void* x;
    const float* dt;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    const void* beta;
    const int32_t* parents;
    const int32_t* last;
    const float* pool;
    const int32_t* slots;
    const int32_t* out;
    const void* y;
};
enum Kind { kStep, kTree, kCommit };

int check(const ssd_pool_problem* p, Kind kind) {
    if (!p) return SSD_ERR_NULL;
    if (p->batch < 0 || p->seqlen < 0 || p->nheads <= 0 || p->headdim <= 0 || p->dstate <= 0 || p->ngroups <= 0 ||
        p->nheads % p->ngroups != 0 || p->slots < 0)
        return SSD_ERR_SHAPE;
    if (p->dtype != SSD_F32 && p->dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (!pn_supported(p->headdim, p->dstate) || p->flags != 0) return SSD_ERR_UNSUPPORTED;
    if (kind != kStep && p->seqlen > SSD_TREE_NODES) return SSD_ERR_UNSUPPORTED;
    const int64_t H = p->nheads, top = (int64_t)1 << 24;
    if (H >= top || p->batch >= top || p->batch * H >= top || H * p->headdim > top) return SSD_ERR_UNSUPPORTED;
    const int64_t state = H * p->headdim * p->dstate;
    if (p->slots > 0x7fffffffLL || state > kFar || p->slot_stride > kFar) return SSD_ERR_UNSUPPORTED;
    if (p->slots > 1 && p->slot_stride < state) return SSD_ERR_SHAPE;
    if (p->slots > 1 && p->slots > ((int64_t)1 << 44) / p->slot_stride) return SSD_ERR_UNSUPPORTED;
    if (p->batch > 0 && p->seqlen > 0) {
        const int64_t most = (int64_t)1 << 32;
        if (p->seqlen > kFar / p->batch) return SSD_ERR_UNSUPPORTED;
        const int64_t tok = p->batch * p->seqlen;
        const int64_t strides[] = {p->xstride, p->bstride, kind == kCommit ? 0 : p->cstride};
        const int64_t rows[] = {H * p->headdim, p->ngroups * p->dstate, kind == kCommit ? 0 : p->ngroups * p->dstate};
        for (int i = 0; i < 3; ++i) {
            if (strides[i] < rows[i]) return SSD_ERR_SHAPE;
            if (strides[i] > most || (strides[i] && tok > kFar / strides[i])) return SSD_ERR_UNSUPPORTED;
        }
        if (H * p->headdim > most || tok > kFar / (H * p->headdim)) return SSD_ERR_UNSUPPORTED;
    }
    return SSD_OK;
}

// Checks a call's operands and enqueues it.
int go(const ssd_pool_problem* p, Kind kind, const Call& c, void* stream) {
    const int st = check(p, kind);
    if (st) return st;
    const int64_t b = p->batch, T = p->seqlen, H = p->nheads, P = p->headdim, N = p->dstate, G = p->ngroups;
    // no rows; no tokens, and no state that goes to another slot
    if (b == 0 || (T == 0 && (kind == kTree || !c.out))) return SSD_OK;
    const bool tree = kind == kTree, commit = kind == kCommit;
    if (!c.slots || (p->slots > 0 && !c.pool) || (commit && !c.last) || !c.A) return SSD_ERR_NULL;
    if (T > 0 && (!c.x || !c.dt || !c.B || (!commit && (!c.C || !c.y)) || (kind != kStep && !c.parents))) return SSD_ERR_NULL;
    if (c.beta && c.D) return SSD_ERR_UNSUPPORTED;
    const size_t es = esize(p->dtype);
    if (!aligned(c.x, 16) || !aligned(c.B, 16) || !aligned(c.C, 16) || !aligned(c.y, 16) || !aligned(c.pool, 16) ||
        !aligned(c.beta, es))
        return SSD_ERR_ALIGN;
    const void* words[] = {c.dt, c.A, c.D, c.parents, c.last, c.slots, c.out};
    for (const void* v : words)
        if (!aligned(v, 4)) return SSD_ERR_ALIGN;
    if ((p->slots > 1 && p->slot_stride % 4 != 0) ||
        (T > 0 && (p->xstride * es % 16 || p->bstride * es % 16 || (!commit && p->cstride * es % 16))))
        return SSD_ERR_ALIGN;
    const int64_t tok = b * T;
    auto span = [&](int64_t stride, int64_t row) { return tok ? (size_t)((tok - 1) * stride + row) * es : 0; };
    const size_t held = p->slots ? (size_t)((p->slots - 1) * (p->slots > 1 ? p->slot_stride : 0) + H * P * N) * 4 : 0;
    const Range rpool = {c.pool, held}, ry = {c.y, (size_t)(tok * H * P) * es};
    const Range ins[] = {{c.x, span(p->xstride, H * P)}, {c.dt, (size_t)(tok * H) * 4}, {c.A, (size_t)H * 4},
                         {c.B, span(p->bstride, G * N)}, {c.C, commit ? (size_t)0 : span(p->cstride, G * N)},
                         {c.D, (size_t)H * 4}, {c.beta, (size_t)(tok * H) * es}, {c.parents, (size_t)tok * 4},
                         {c.last, (size_t)b * 4}, {c.slots, (size_t)b * 4}, {c.out, (size_t)b * 4}};
    const Range outs[] = {tree ? Range{nullptr, 0} : rpool, ry};
    if (any_overlap(outs, 2, ins, 11) || overlap(ry, rpool)) return SSD_ERR_ALIAS;

    Args a;
    memset(&a, 0, sizeof(a));
    a.b = b; a.T = T; a.H = (int)H; a.P = (int)P; a.N = (int)N; a.G = (int)G;
    a.xs = p->xstride; a.bs = p->bstride; a.cs = p->cstride;
    a.S = p->slots; a.ss = p->slots > 1 ? p->slot_stride : 0;
    a.x = c.x; a.dt = c.dt; a.A = c.A; a.B = c.B; a.C = c.C; a.D = c.D; a.beta = c.beta;
    a.parents = c.parents; a.last = c.last;
    a.pool = const_cast<float*>(c.pool);
    a.slots = c.slots;
    a.out = c.out ? c.out : c.slots;
    a.y = const_cast<void*>(c.y);
    a.stream = (hipStream_t)stream;
    const bool half = p->dtype == SSD_BF16;
    if (tree) return half ? ssd::pool::tree_bf16(a) : ssd::pool::tree_f32(a);
    return half ? ssd::pool::run_walk<ssd::bf16>(a, commit) : ssd::pool::run_walk<float>(a, commit);
}

// ---- the pool's pages ----
int check_pages(const ssd_pages* p, bool fork) {
    if (!p) return SSD_ERR_NULL;
    if (p->rows < 0 || p->layers < 0 || p->slots < 0 || p->slot_elems <= 0) return SSD_ERR_SHAPE;
    if (fork && p->rows > p->slots) return SSD_ERR_SHAPE;
    if (p->rows > 65536 || p->slots > ssd::pool::kSlots || p->layers > 65536 || p->slot_elems > kFar)
        return SSD_ERR_UNSUPPORTED;
    const bool ls = p->layers > 1, ss = p->slots > 1;  // (a stride of one layer or slot is not used)
    if ((ls && p->layer_stride < p->slot_elems) || (ss && p->slot_stride < p->slot_elems)) return SSD_ERR_SHAPE;
    if ((ls && p->layer_stride > kFar) || (ss && p->slot_stride > kFar)) return SSD_ERR_UNSUPPORTED;
    // layers of whole slots, or slots of whole layers
    if (ls && ss && p->layer_stride < (p->slots - 1) * p->slot_stride + p->slot_elems &&
        p->slot_stride < (p->layers - 1) * p->layer_stride + p->slot_elems)
        return SSD_ERR_SHAPE;
    return SSD_OK;
}

int pages(const ssd_pages* p, bool fork, float* pool, const int32_t* table, const int32_t* sources, int32_t* fresh,
          int32_t* count, void* stream) {
    const int st = check_pages(p, fork);
    if (st) return st;
    if (p->rows == 0 && fork) return SSD_OK;
    if ((p->rows > 0 && (!table || !fresh)) || (fork && !sources) || (!fork && !count)) return SSD_ERR_NULL;
    if (!pool && p->layers > 0 && p->slots > 0) return SSD_ERR_NULL;
    const bool ls = p->layers > 1, ss = p->slots > 1;
    if (!aligned(pool, 16) || p->slot_elems % 4 || (ls && p->layer_stride % 4) || (ss && p->slot_stride % 4) ||
        !aligned(table, 4) || !aligned(sources, 4) || !aligned(fresh, 4) || !aligned(count, 4))
        return SSD_ERR_ALIGN;
    const size_t held = p->layers && p->slots
                            ? (size_t)((ls ? (p->layers - 1) * p->layer_stride : 0) +
                                       (ss ? (p->slots - 1) * p->slot_stride : 0) + p->slot_elems) * 4
                            : 0;
    const size_t rows = (size_t)p->rows * 4;
    const Range ins[] = {{table, rows}, {sources, fork ? rows : (size_t)0}};
    const Range outs[] = {{pool, held}, {fresh, rows}, {count, (size_t)(fork ? 0 : 4)}};
    if (any_overlap(outs, 3, ins, 2)) return SSD_ERR_ALIAS;

    ssd::pool::PageArgs a;
    memset(&a, 0, sizeof(a));
    a.layers = p->layers; a.elems = p->slot_elems;
    a.ls = ls ? p->layer_stride : 0; a.ss = ss ? p->slot_stride : 0;
    a.R = (int)p->rows; a.S = (int)p->slots;
    a.pool = pool; a.table = table; a.sources = sources; a.fresh = fresh; a.count = count;
    a.stream = (hipStream_t)stream;
    const size_t lds = fork ? ssd::pool::fork_lds(a.R, a.S) : ssd::pool::compact_lds(a.S);
    const int64_t moves = fork ? p->rows : (p->rows < p->slots / 2 ? p->rows : p->slots / 2);
    const unsigned grid = ssd::pool::page_grid(a, moves, lds);
    if (lds > 64 * 1024 && hipFuncSetAttribute((const void*)ssd::pool::k_fork, hipFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)lds) != hipSuccess)
        return SSD_ERR_HIP;
    if (fork) ssd::pool::k_fork<<<grid, 256, lds, a.stream>>>(a);
    else ssd::pool::k_compact<<<grid, 256, lds, a.stream>>>(a);
    return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

}  // namespace

extern "C" {

int ssd_pool_step(const ssd_pool_problem* p, const void* x, const float* dt, const float* A, const void* B,
                  const void* C, const float* D, const void* beta, float* pool, const int32_t* slots,
                  const int32_t* out_slots, void* y, void* stream) {
    return go(p, kStep, {x, dt, A, B, C, D, beta, nullptr, nullptr, pool, slots, out_slots, y}, stream);
}

int ssd_tree_step(const ssd_pool_problem* p, const void* x, const float* dt, const float* A, const void* B,
                  const void* C, const float* D, const void* beta, const int32_t* parents, const float* pool,
                  const int32_t* slots, void* y, void* stream) {
    return go(p, kTree, {x, dt, A, B, C, D, beta, parents, nullptr, pool, slots, nullptr, y}, stream);
}

int ssd_tree_commit(const ssd_pool_problem* p, const void* x, const float* dt, const float* A, const void* B,
                    const void* beta, const int32_t* parents, const int32_t* last, float* pool,
                    const int32_t* slots, const int32_t* out_slots, void* stream) {
    return go(p, kCommit, {x, dt, A, B, nullptr, nullptr, beta, parents, last, pool, slots, out_slots, nullptr}, stream);
}

int ssd_pool_fork(const ssd_pages* p, float* pool, const int32_t* table, const int32_t* sources, int32_t* new_table,
                  void* stream) {
    return pages(p, true, pool, table, sources, new_table, nullptr, stream);
}

int ssd_pool_compact(const ssd_pages* p, float* pool, const int32_t* table, int32_t* new_table, int32_t* count,
                     void* stream) {
    return pages(p, false, pool, table, nullptr, new_table, count, stream);
}

}  // extern "C"
