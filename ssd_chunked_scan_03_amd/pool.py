"""States of many sequences in a pool: the decode step through slot indices, trees of drafted tokens
over the held states, and the pool's pages.

    y = pool_step(x, dt, A, B, C, pool, slots, D=None, beta=None, out_slots=None)
    y = tree_step(x, dt, A, B, C, parents, pool, slots, D=None, beta=None)
    tree_commit(x, dt, A, B, parents, last, pool, slots, beta=None, out_slots=None)
    table = pool_fork(pool, table, sources)
    table, count = pool_compact(pool, table)

pool [S, H, P, N] f32 holds one state per slot (for pool_fork and pool_compact also [L, S, H, P, N],
all layers at once; ``pool[l]`` is one layer's pool); slots [b] int32 names the slot of every row, and a
row whose slot is outside [0, S) is idle (its y is zero).  x, B and C may be views into a wider projection
(heads contiguous, tokens evenly spaced).  ``beta`` [b, T, H] selects the gated delta rule; without it the
scan's recurrence runs, with its skip term D.  No slot may be written by one row and read or written by
another row of the same call.
"""
from __future__ import annotations

import ctypes
import functools

from .delta import _call, _codes, _token_stride

TREE_NODES = 256


class PoolProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("batch", "seqlen", "nheads", "headdim", "dstate", "ngroups", "xstride", "bstride", "cstride", "slots",
                 "slot_stride")] + [("dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


class Pages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("rows", "layers", "slots", "slot_elems", "layer_stride", "slot_stride")]


def _bind(lib):
    """Argument types of this module's entry points."""
    P, Q = ctypes.POINTER(PoolProblem), ctypes.POINTER(Pages)
    vp, ci = ctypes.c_void_p, ctypes.c_int
    for name, args in (("ssd_pool_step", [P] + [vp] * 12), ("ssd_tree_step", [P] + [vp] * 12),
                       ("ssd_tree_commit", [P] + [vp] * 11), ("ssd_pool_fork", [Q] + [vp] * 5),
                       ("ssd_pool_compact", [Q] + [vp] * 5)):
        f = getattr(lib, name)
        f.restype, f.argtypes = ci, args


@functools.lru_cache(maxsize=256)
def _pages(*sizes):
    return Pages(*sizes)


def _refuse(x, tensors):
    """The message of the first of (name, tensor, shape, dtype) that is not as it has to be."""
    for name, t, shape, dtype in tensors:
        if t is None:
            continue
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_cuda or t.device != x.device:
            raise ValueError(f"{name} must be a GPU tensor on {x.device}, where x is")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _slot_stride(pool):
    """Elements from one slot to the next of a [S, H, P, N] pool whose slots are whole."""
    S, H, P, N = pool.shape
    if pool.is_contiguous():
        return H * P * N
    if pool.stride(3) != 1 or (P > 1 and pool.stride(2) != N) or (H > 1 and pool.stride(1) != P * N):
        raise ValueError("each slot of pool must be contiguous")
    return pool.stride(0) if S > 1 else H * P * N


# Sizes, strides, type and device of a call's x, B, C and pool (no data) -> its descriptor, the device and what
# its other tensors have to be, so that these are worked out once for each.
_seen = {}
_OTHERS = {"step": ("dt", "A", "D", "beta", "slots", "out_slots"), "tree": ("dt", "A", "D", "beta", "parents", "slots"),
           "commit": ("dt", "A", "beta", "parents", "last", "slots", "out_slots")}


def _rows(kind, x, B, C, pool, others):
    """Checks a call's tensors (others: in _OTHERS' order) and returns its descriptor and device."""
    if others[-1 if kind == "tree" else -2] is None:
        raise ValueError("slots is required")
    look = (kind, x.shape, x.stride(), x.dtype, x.get_device(), B.shape, B.stride(), pool.shape, pool.stride(),
            None if C is None else C.stride())
    found = _seen.get(look)
    if found is None:
        found = _work_out(kind, x, B, C, pool)
        if len(_seen) >= 1024:
            _seen.clear()
        _seen[look] = found
    prob, dev, want = found
    td, ok = x.dtype, B.dtype == x.dtype and B.get_device() == dev and pool.get_device() == dev
    if C is not None:
        ok = ok and C.dtype == td and C.get_device() == dev and C.shape == B.shape
    for t, (shape, dtype) in zip(others, want):
        if t is not None and (t.shape != shape or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous()):
            ok = False
    if not ok or pool.dtype != want[0][1]:  # (dt's type: float32)
        _work_out(kind, x, B, C, pool)
        _refuse(x, [(n, t, *w) for n, t, w in zip(_OTHERS[kind], others, want)])
    if kind != "commit" and others[2] is not None and others[3] is not None:
        raise ValueError("the gated delta rule (beta) has no skip term D")
    return prob, dev


def _work_out(kind, x, B, C, pool):
    import torch
    if x.dim() != 4 or B.dim() != 4 or pool.dim() != 4:
        raise ValueError("x must be [b, T, H, P], B [b, T, G, N] and pool [S, H, P, N]")
    b, T, H, P = x.shape
    G, N = B.shape[2:]
    td, f32, i32 = x.dtype, torch.float32, torch.int32
    code = _codes().get(td)
    if code is None:
        raise TypeError(f"x/B/C must be bfloat16 or float32, got {td}")
    dev = x.get_device()
    if pool.shape[1:] != (H, P, N):
        raise ValueError(f"pool must have shape [S, {H}, {P}, {N}], got {tuple(pool.shape)}")
    if pool.dtype != f32:
        raise TypeError(f"pool must be float32, got {pool.dtype}")
    for name, t in (("B", B), ("C", C)):
        if t is not None and t.shape != (b, T, G, N):
            raise ValueError(f"{name} must have shape {(b, T, G, N)}, got {tuple(t.shape)}")
        if t is not None and t.dtype != td:
            raise TypeError("x, B, C must share one dtype")
    if dev < 0 or pool.get_device() != dev or B.get_device() != dev or (C is not None and C.get_device() != dev):
        raise ValueError("x, B, C and pool must be GPU tensors on one device")
    if kind != "step" and T > TREE_NODES:
        raise ValueError(f"a tree has at most {TREE_NODES} nodes, got {T}")
    xs, bs = _step("x", x, T, H, P), _step("B", B, T, G, N)
    cs = 0 if C is None else _step("C", C, T, G, N)
    prob = PoolProblem(b, T, H, P, N, G, xs, bs, cs, pool.shape[0], _slot_stride(pool), code, 0)
    shapes = {"dt": ((b, T, H), f32), "A": ((H,), f32), "D": ((H,), f32), "beta": ((b, T, H), td),
              "parents": ((b, T), i32), "last": ((b,), i32), "slots": ((b,), i32), "out_slots": ((b,), i32)}
    return prob, dev, tuple(shapes[n] for n in _OTHERS[kind])


def _step(name, t, T, heads, n):
    """Elements from one token to the next."""
    s = t.stride()
    step = s[1]
    if T > 1 and s[3] == 1 and s[2] == n and s[0] == T * step and step >= heads * n:
        return step
    return heads * n if t.is_contiguous() else _token_stride(name, t)


def _like(x):
    import torch
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def pool_step_into(prob: PoolProblem, x, dt, A, B, C, D, beta, pool, slots, out_slots, y, stream=None) -> None:
    """Enqueue the recurrence over prob.seqlen tokens of every row: the pool is updated, y receives the
    outputs (no allocation)."""
    _call("ssd_pool_step", prob, (x, dt, A, B, C, D, beta, pool, slots, out_slots, y), stream=stream)


def pool_step(x, dt, A, B, C, pool, slots, D=None, beta=None, out_slots=None):
    """Decode: run the recurrence over x's tokens [b, T, H, P] on the states pool[slots[i]], left in
    pool[out_slots[i]] (None: in place; an out slot outside the pool leaves none).  dt [b, T, H] f32, A and D
    [H] f32, B/C [b, T, G, N], beta [b, T, H] in x's dtype (the gated delta rule, no D) or None.  Returns y."""
    prob, dev = _rows("step", x, B, C, pool, (dt, A, D, beta, slots, out_slots))
    y = _like(x)
    _call("ssd_pool_step", prob, (x, dt, A, B, C, D, beta, pool, slots, out_slots, y), index=dev)
    return y


def tree_step_into(prob: PoolProblem, x, dt, A, B, C, D, beta, parents, pool, slots, y, stream=None) -> None:
    """Enqueue one pass over the trees (prob.seqlen nodes a row) into y (no allocation)."""
    _call("ssd_tree_step", prob, (x, dt, A, B, C, D, beta, parents, pool, slots, y), stream=stream)


def tree_step(x, dt, A, B, C, parents, pool, slots, D=None, beta=None):
    """A tree of drafted tokens over the held states: x [b, K, H, P], dt [b, K, H], B/C [b, K, G, N],
    beta [b, K, H] or None; parents [b, K] int32, each a node before it or -1 (the held state pool[slots[i]]).  A
    node with any other parent, or below such a node, is absent: pad rows of fewer nodes with -2.  K is
    at most 256.  Returns y [b, K, H, P] (zero for absent nodes); the pool is left as it is."""
    prob, dev = _rows("tree", x, B, C, pool, (dt, A, D, beta, parents, slots))
    y = _like(x)
    _call("ssd_tree_step", prob, (x, dt, A, B, C, D, beta, parents, pool, slots, y), index=dev)
    return y


def tree_commit_into(prob: PoolProblem, x, dt, A, B, beta, parents, last, pool, slots, out_slots, stream=None) -> None:
    """Enqueue the commit of one node of every row's tree into the pool (no allocation)."""
    _call("ssd_tree_commit", prob, (x, dt, A, B, beta, parents, last, pool, slots, out_slots), stream=stream)


def tree_commit(x, dt, A, B, parents, last, pool, slots, beta=None, out_slots=None):
    """Accept a path of tree_step's tree (same arguments): the state behind node last[i] (int32 [b]; -1: the
    held state itself) goes to pool[out_slots[i]] (None: in place).  Returns the pool."""
    prob, dev = _rows("commit", x, B, None, pool, (dt, A, beta, parents, last, slots, out_slots))
    _call("ssd_tree_commit", prob, (x, dt, A, B, beta, parents, last, pool, slots, out_slots), index=dev)
    return pool


# ---- the pool's pages ----
def _layout(pool, table, sources=None):
    import torch
    if pool.dim() not in (4, 5):
        raise ValueError("pool must be [S, H, P, N] or [L, S, H, P, N]")
    if pool.dtype != torch.float32:
        raise TypeError(f"pool must be float32, got {pool.dtype}")
    H, P, N = pool.shape[-3:]
    elems, S = H * P * N, pool.shape[-4]
    L = pool.shape[0] if pool.dim() == 5 else 1
    ss, ls = pool.stride(-4), pool.stride(0)
    if not pool.is_contiguous() and pool.numel():
        if ((N > 1 and pool.stride(-1) != 1) or (P > 1 and pool.stride(-2) != N) or (H > 1 and pool.stride(-3) != P * N)):
            raise ValueError("each slot of pool must be contiguous")
    dev = pool.get_device()
    if dev < 0:
        raise ValueError("pool must be a GPU tensor")
    if table.dim() != 1:
        raise ValueError("table must be [rows]")
    for name, t in (("table", table), ("sources", sources)):
        if t is None:
            continue
        if t.shape != table.shape:
            raise ValueError(f"{name} must have shape {tuple(table.shape)}, got {tuple(t.shape)}")
        if t.dtype != torch.int32:
            raise TypeError(f"{name} must be int32, got {t.dtype}")
        if t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous and on pool's device")
    R = table.shape[0]
    if sources is not None and R > S:
        raise ValueError(f"a table of {R} rows needs a pool of as many slots, got {S}")
    return _pages(R, L, S, elems, ls if L > 1 else 0, ss if S > 1 else 0)


def pool_fork_into(prob: Pages, pool, table, sources, new_table, stream=None) -> None:
    """Enqueue one fork: the pool is updated, new_table receives the rows' slots (no allocation)."""
    _call("ssd_pool_fork", prob, (pool, table, sources, new_table), stream=stream)


def pool_fork(pool, table, sources):
    """Fork, free and begin sequences: table [R] int32 names every row's slot (outside [0, S): none); in the
    returned table row r goes on from row sources[r] of the old one (int32 [R]), is freed (-1), or begins from
    a zero state (-2).  One row takes a slot over, the others get copies in free slots; R is at most S."""
    import torch
    if sources is None:
        raise ValueError("sources is required")
    prob = _layout(pool, table, sources)
    new = torch.empty_like(table)
    _call("ssd_pool_fork", prob, (pool, table, sources, new), index=pool.get_device())
    return new


def pool_compact_into(prob: Pages, pool, table, new_table, count, stream=None) -> None:
    """Enqueue one compaction: the pool is updated, new_table receives the rows' slots and count [1] the
    number of slots in use (no allocation)."""
    _call("ssd_pool_compact", prob, (pool, table, new_table, count), stream=stream)


def pool_compact(pool, table):
    """Bring the slots that table [R] (int32; outside [0, S): none) names to the front: of n named slots those
    from n on move into unnamed ones below n.  Returns (new table, count): count [1] int32 holds n on the
    device, so that pool[:n] is a contiguous batch of states."""
    import torch
    prob = _layout(pool, table)
    new = torch.empty_like(table)
    count = torch.empty(1, dtype=torch.int32, device=pool.device)
    _call("ssd_pool_compact", prob, (pool, table, new, count), index=pool.get_device())
    return new, count
