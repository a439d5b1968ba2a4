"""The gated delta rule on the scan's operands, and the norm of B and C that prepares them.

    y, hT = delta_fwd(x, dt, A, B, C, beta, h0=None)
    y, hT = delta_fwd_varlen(x, dt, A, B, C, beta, cu_seqlens, h0=None)
    y = delta_step(x, dt, A, B, C, beta, h)                     # h updated in place
    grads = delta_bwd(x, dt, A, B, C, beta, dy, h0=None, dhT=None)
    Bn, Cn = bc_norm(B, C, wB=None, wC=None, mode="rms", inv_freq=None, positions=None)
    grads = bc_norm_bwd(B, C, dBn, dCn, wB=None, wC=None, ...)

Layouts as for the scan, with beta [b,T,H] (the write strength) in x's dtype:
r_t = x_t - a_t h_{t-1} B_t, h_t = a_t h_{t-1} + beta_t r_t B_t^T, y_t = h_t C_t,
a_t = exp(dt_t A_h).  Keys are meant to have about unit length; ``norm`` (a dict of
:func:`bc_norm`'s keyword arguments) passes B and C through bc_norm first.
"""
from __future__ import annotations

import ctypes
import functools

from . import SSD_BF16, SSD_F32, Problem, SSDError, _check_args, _load, make_problem

DELTA_CHUNK = 64
NORM_MODES = {"rms": 0, "l2": 1}


class Norm(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("bheads", ctypes.c_int64),
                ("cheads", ctypes.c_int64), ("dstate", ctypes.c_int64), ("pairs", ctypes.c_int64),
                ("bstride", ctypes.c_int64), ("cstride", ctypes.c_int64), ("eps", ctypes.c_float),
                ("mode", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("dtype", ctypes.c_int32)]


def _bind(lib):
    """Argument types of this module's entry points."""
    P, Q = ctypes.POINTER(Problem), ctypes.POINTER(Norm)
    vp, sz, ci = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    for name, res, args in (
            ("ssd_delta_workspace_bytes", sz, [P]), ("ssd_delta_varlen_workspace_bytes", sz, [P]),
            ("ssd_delta_bwd_workspace_bytes", sz, [P]), ("ssd_bc_norm_bwd_workspace_bytes", sz, [Q]),
            ("ssd_delta_fwd", ci, [P] + [vp] * 10 + [sz, vp]),
            ("ssd_delta_fwd_varlen", ci, [P] + [vp] * 11 + [sz, vp]),
            ("ssd_delta_step", ci, [P] + [vp] * 9),
            ("ssd_delta_bwd", ci, [P] + [vp] * 17 + [sz, vp]),
            ("ssd_bc_norm", ci, [Q] + [vp] * 9),
            ("ssd_bc_norm_bwd", ci, [Q] + [vp] * 13 + [sz, vp])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args


_calls = {}  # bound entry points


def _raw_stream(index):
    """The current stream of device `index` as an integer (hipStream_t)."""
    import torch
    f = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return f(index) if f is not None else torch.cuda.current_stream(index).cuda_stream


def _call(name, head, tensors, ws=False, stream=None, index=None):
    """Enqueue one entry point on `stream` (default: the current stream of the tensors' device,
    which the call makes the current device meanwhile).  All of `tensors` and the workspace `ws`
    (False: the entry point takes none) lie on that one GPU, `index` where the caller has checked
    them: a kernel would read a host address."""
    import torch
    fn = _calls.get(name)
    if fn is None:
        fn = _calls[name] = getattr(_load(), name)
    if index is None:
        on = {t.get_device() for t in (*tensors, None if ws is False else ws) if t is not None}
        index = on.pop() if len(on) == 1 else -1
        if index < 0:
            raise ValueError(f"{name} needs GPU tensors, all on one device")
    args = [None if t is None else t.data_ptr() for t in tensors]
    if ws is not False:
        args += (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())
    if index == torch.cuda.current_device():
        st = fn(head, *args, _raw_stream(index) if stream is None else int(stream))
    else:
        with torch.cuda.device(index):
            st = fn(head, *args, _raw_stream(index) if stream is None else int(stream))
    if st:
        raise SSDError(st, name)


@functools.lru_cache(maxsize=256)
def _plan(kind, b, T, H, P, N, G, chunk, code):
    """The problem of these sizes and its workspace bytes (a descriptor: it holds no data)."""
    prob = make_problem(b, T, H, P, N, G, chunk, code)
    return prob, (0 if kind == "step" else delta_bwd_workspace_bytes(prob) if kind == "bwd"
                  else delta_workspace_bytes(prob, kind == "varlen"))


def _check(x, tensors):
    """_check_args for (name, tensor or None, shape, dtype) entries against x's device; the
    message is formed only where something is wrong."""
    dev = x.get_device()
    ok = dev >= 0 and x.dtype in _codes()
    for _, t, shape, dtype in tensors:
        if t is not None and (t.shape != shape or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous()):
            ok = False
    if not ok:
        import torch
        _check_args({n: (t, shape) for n, t, shape, _ in tensors},
                    floats=[n for n, _, _, d in tensors if d == torch.float32 and n not in _PROBLEM_DTYPE],
                    same_dtype=[n for n, t, _, _ in tensors if n in _PROBLEM_DTYPE])
        for n, t, _, dtype in tensors:
            if t is not None and t.dtype != dtype:
                raise TypeError(f"{n} must be {dtype}, got {t.dtype}")
    return _codes()[x.dtype]


_PROBLEM_DTYPE = ("x", "B", "C", "beta", "dy")


@functools.lru_cache(maxsize=1)
def _codes():
    import torch
    return {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16}


def delta_workspace_bytes(prob: Problem, varlen: bool = False) -> int:
    lib = _load()
    f = lib.ssd_delta_varlen_workspace_bytes if varlen else lib.ssd_delta_workspace_bytes
    return int(f(ctypes.byref(prob)))


def delta_bwd_workspace_bytes(prob: Problem) -> int:
    return int(_load().ssd_delta_bwd_workspace_bytes(ctypes.byref(prob)))


def _workspace(ws, need, device):
    import torch
    if ws is not None and ws.device != device:
        raise ValueError(f"workspace is on {ws.device}, the other tensors on {device}")
    if ws is None or ws.numel() * ws.element_size() < need:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    return ws


def delta_fwd_into(prob: Problem, x, dt, A, B, C, beta, h0, y, hT, ws, stream=None) -> None:
    """Enqueue one forward into caller-provided outputs and workspace (no allocation)."""
    _call("ssd_delta_fwd", prob, (x, dt, A, B, C, beta, h0, y, hT), ws, stream)


def delta_fwd_varlen_into(prob: Problem, cu_seqlens, x, dt, A, B, C, beta, h0, y, hT, ws, stream=None) -> None:
    """Enqueue one packed forward (prob.batch sequences on one axis of prob.seqlen tokens)
    into caller-provided outputs and workspace (no allocation)."""
    _call("ssd_delta_fwd_varlen", prob, (cu_seqlens, x, dt, A, B, C, beta, h0, y, hT), ws, stream)


def delta_step_into(prob: Problem, x, dt, A, B, C, beta, h, y, stream=None) -> None:
    """Enqueue the rule over prob.seqlen tokens: h is updated in place, y receives the
    outputs (no allocation)."""
    _call("ssd_delta_step", prob, (x, dt, A, B, C, beta, h, y), stream=stream)


def delta_bwd_into(prob: Problem, x, dt, A, B, C, beta, h0, dy, dhT, dx, ddt, dA, dB, dC, dbeta, dh0, ws,
                   stream=None) -> None:
    """Enqueue one backward pass into caller-provided gradients and workspace (no allocation)."""
    _call("ssd_delta_bwd", prob, (x, dt, A, B, C, beta, h0, dy, dhT, dx, ddt, dA, dB, dC, dbeta, dh0), ws, stream)


def _normed(B, C, norm):
    return (B, C) if norm is None else bc_norm(B, C, **norm)


def _shapes4(x, B):
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [b, T, H, P] and B [b, T, G, N]")
    return (*x.shape, B.shape[2], B.shape[3])


def delta_fwd(x, dt, A, B, C, beta, h0=None, chunk=DELTA_CHUNK, return_final_state=True, workspace=None, norm=None):
    """Gated delta rule forward: x [b, T, H, P], dt [b, T, H] f32, A [H] f32, B/C [b, T, G, N],
    beta [b, T, H] in x's dtype, h0 [b, H, P, N] f32 or None.  A ``norm`` that turns counts the
    tokens from 0: where h0 is the state behind earlier tokens, give it their positions.
    Returns (y, hT)."""
    import torch
    b, T, H, P, G, N = _shapes4(x, B)
    B, C = _normed(B, C, norm)
    f32, td = torch.float32, x.dtype
    code = _check(x, (("x", x, (b, T, H, P), td), ("dt", dt, (b, T, H), f32), ("A", A, (H,), f32),
                      ("B", B, (b, T, G, N), td), ("C", C, (b, T, G, N), td), ("beta", beta, (b, T, H), td),
                      ("h0", h0, (b, H, P, N), f32)))
    prob, need = _plan("fwd", b, T, H, P, N, G, chunk, code)
    y = torch.empty_like(x)
    hT = torch.empty((b, H, P, N), dtype=f32, device=x.device) if return_final_state else None
    _call("ssd_delta_fwd", prob, (x, dt, A, B, C, beta, h0, y, hT), _workspace(workspace, need, x.device),
          index=x.get_device())
    return y, hT


def delta_fwd_varlen(x, dt, A, B, C, beta, cu_seqlens, h0=None, chunk=DELTA_CHUNK, return_final_state=True,
                     workspace=None, norm=None):
    """Gated delta rule forward over packed sequences: x [T, H, P], dt [T, H], B/C [T, G, N],
    beta [T, H]; sequence s on tokens [cu_seqlens[s], cu_seqlens[s+1]) (int32 GPU tensor);
    h0 / hT [nseq, H, P, N].  Rows of y outside every sequence are not written.  Returns
    (y, hT)."""
    import torch
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise TypeError("cu_seqlens must be a 1-D int32 tensor of nseq + 1 offsets")
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [T, H, P] and B [T, G, N]")
    T, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    nseq = cu_seqlens.numel() - 1
    if norm is not None:
        if norm.get("inv_freq") is not None and norm.get("positions") is None:
            raise ValueError("packed sequences need norm's positions: every sequence counts its own")
        pos = norm.get("positions")
        Bn, Cn = bc_norm(B[None], C[None], **dict(norm, positions=None if pos is None else pos.reshape(1, -1)))
        B, C = Bn[0], Cn[0]
    f32, td = torch.float32, x.dtype
    code = _check(x, (("x", x, (T, H, P), td), ("dt", dt, (T, H), f32), ("A", A, (H,), f32), ("B", B, (T, G, N), td),
                      ("C", C, (T, G, N), td), ("beta", beta, (T, H), td), ("h0", h0, (nseq, H, P, N), f32),
                      ("cu_seqlens", cu_seqlens, (nseq + 1,), torch.int32)))
    prob, need = _plan("varlen", nseq, T, H, P, N, G, chunk, code)
    y = torch.empty_like(x)
    hT = torch.empty((nseq, H, P, N), dtype=f32, device=x.device) if return_final_state else None
    _call("ssd_delta_fwd_varlen", prob, (cu_seqlens, x, dt, A, B, C, beta, h0, y, hT),
          _workspace(workspace, need, x.device), index=x.get_device())
    return y, hT


def delta_step(x, dt, A, B, C, beta, h, norm=None):
    """Decode: run the rule over x's tokens on state h [b, H, P, N] f32 (updated in place).
    x [b, T, H, P], dt [b, T, H] f32, A [H] f32, B/C [b, T, G, N], beta [b, T, H].  Returns y.
    A ``norm`` that turns (inv_freq) needs the tokens' positions behind what h has seen: without
    them the call's tokens count from 0, which only the first tokens of an empty state do, so a
    single token is refused."""
    import torch
    b, T, H, P, G, N = _shapes4(x, B)
    if h is None:
        raise ValueError("h (the state, updated in place) is required")
    if T == 1 and norm is not None and norm.get("inv_freq") is not None and norm.get("positions") is None:
        raise ValueError("a decode step needs norm's positions: its token is not the sequence's first")
    B, C = _normed(B, C, norm)
    f32, td = torch.float32, x.dtype
    code = _check(x, (("x", x, (b, T, H, P), td), ("dt", dt, (b, T, H), f32), ("A", A, (H,), f32),
                      ("B", B, (b, T, G, N), td), ("C", C, (b, T, G, N), td), ("beta", beta, (b, T, H), td),
                      ("h", h, (b, H, P, N), f32)))
    prob, _ = _plan("step", b, T, H, P, N, G, DELTA_CHUNK, code)
    y = torch.empty_like(x)
    _call("ssd_delta_step", prob, (x, dt, A, B, C, beta, h, y), index=x.get_device())
    return y


def delta_bwd(x, dt, A, B, C, beta, dy, h0=None, dhT=None, chunk=DELTA_CHUNK, workspace=None, norm=None):
    """Backward pass of delta_fwd: gradients of a loss with respect to every input, given dy
    (like x) and dhT ([b, H, P, N] float32, None = 0).  Returns a dict with dx, dB, dC, dbeta
    (their inputs' dtype), ddt, dA and dh0 (float32).  With ``norm``, dB and dC are the
    gradients of the tensors before bc_norm, and dwB / dwC are added for its weights."""
    import torch
    b, T, H, P, G, N = _shapes4(x, B)
    B0, C0 = B, C
    B, C = _normed(B, C, norm)
    f32, td = torch.float32, x.dtype
    code = _check(x, (("x", x, (b, T, H, P), td), ("dt", dt, (b, T, H), f32), ("A", A, (H,), f32),
                      ("B", B, (b, T, G, N), td), ("C", C, (b, T, G, N), td), ("beta", beta, (b, T, H), td),
                      ("dy", dy, (b, T, H, P), td), ("h0", h0, (b, H, P, N), f32), ("dhT", dhT, (b, H, P, N), f32)))
    prob, need = _plan("bwd", b, T, H, P, N, G, chunk, code)
    e = torch.empty_like
    out = dict(dx=e(x), ddt=e(dt), dA=e(A), dB=e(B), dC=e(C), dbeta=e(beta),
               dh0=torch.empty((b, H, P, N), dtype=f32, device=x.device))
    _call("ssd_delta_bwd", prob, (x, dt, A, B, C, beta, h0, dy, dhT, *out.values()),
          _workspace(workspace, need, x.device), index=x.get_device())
    if norm is not None:
        out.update(bc_norm_bwd(B0, C0, out["dB"], out["dC"], **norm))
    return out


# ---- the norm of B and C ----
def _token_stride(name, t):
    """Elements between tokens of a [b, T, heads, N] tensor whose heads are contiguous; views
    into a wider projection are accepted as they are."""
    b, T, heads, N = t.shape
    if t.numel() == 0:
        return heads * N
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.stride(3) != 1 or (heads > 1 and t.stride(2) != N):
        raise ValueError(f"{name}'s heads must be contiguous")
    if T > 1:
        step = t.stride(1)
        if b > 1 and t.stride(0) != T * step:
            raise ValueError(f"{name}'s tokens must be evenly spaced over the batch")
    else:
        step = t.stride(0) if b > 1 else heads * N
    if step < heads * N:
        raise ValueError(f"{name}'s tokens must not overlap")
    return step


@functools.lru_cache(maxsize=256)
def _norm_plan(*sizes):
    """The descriptor of these sizes and its backward's workspace bytes."""
    prob = Norm(*sizes)
    return prob, bc_norm_bwd_workspace_bytes(prob)


def _norm_problem(B, C, wB, wC, mode, eps, inv_freq, positions, interleaved):
    import torch
    if B.dim() != 4 or C.dim() != 4:
        raise ValueError("B and C must be [b, T, heads, N]")
    b, T, GB, N = B.shape
    GC = C.shape[2]
    if mode not in NORM_MODES:
        raise ValueError(f"mode must be one of {sorted(NORM_MODES)}, got {mode!r}")
    if C.shape != (b, T, GC, N):
        raise ValueError(f"C must have shape {(b, T, GC, N)}, got {tuple(C.shape)}")
    F = 0 if inv_freq is None else inv_freq.numel()
    code = _codes().get(B.dtype)
    if code is None:
        raise TypeError(f"B and C must be bfloat16 or float32, got {B.dtype}")
    if C.dtype != B.dtype:
        raise TypeError("B, C must share one dtype")
    dev, f32 = B.get_device(), torch.float32
    for t, shape, dtype in ((wB, (N,), f32), (wC, (N,), f32), (inv_freq, (F,), f32), (positions, (b, T), torch.int32)):
        if t is not None and (t.shape != shape or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous()):
            name = "wB" if t is wB else "wC" if t is wC else "inv_freq" if t is inv_freq else "positions"
            _norm_refuse(t, name, shape, dtype, B)
    if dev < 0 or C.get_device() != dev:
        raise ValueError("B and C must be GPU tensors on one device")
    sB = GB * N if B.is_contiguous() else _token_stride("B", B)
    sC = GC * N if C.is_contiguous() else _token_stride("C", C)
    return _norm_plan(b, T, GB, GC, N, F, sB, sC, float(eps), NORM_MODES[mode], int(bool(interleaved)), code)


def _norm_refuse(t, name, shape, dtype, B):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be a contiguous tensor on {B.device}")


def bc_norm_into(prob: Norm, B, C, wB, wC, inv_freq, positions, Bn, Cn, stream=None) -> None:
    """Enqueue one norm into caller-provided outputs (no allocation)."""
    _call("ssd_bc_norm", prob, (B, C, wB, wC, inv_freq, positions, Bn, Cn), stream=stream)


def bc_norm(B, C, wB=None, wC=None, mode="rms", eps=1e-6, inv_freq=None, positions=None, interleaved=False):
    """Normalise every head's row of B [b, T, GB, N] and C [b, T, GC, N] (rms or l2), scale by
    the weights wB / wC ([N] f32) and turn it by its position: pairs (i, i + F), or
    (2i, 2i + 1) where interleaved, by positions [b, T] (int32; default: the token's index)
    times inv_freq [F] (f32, F a multiple of 4, 2F <= N; None: no rotation).  B and C may be
    views into a wider projection.  Returns (Bn, Cn), contiguous."""
    import torch
    prob, _ = _norm_problem(B, C, wB, wC, mode, eps, inv_freq, positions, interleaved)
    whole = torch.contiguous_format
    Bn, Cn = torch.empty_like(B, memory_format=whole), torch.empty_like(C, memory_format=whole)
    _call("ssd_bc_norm", prob, (B, C, wB, wC, inv_freq, positions, Bn, Cn), index=B.get_device())
    return Bn, Cn


def bc_norm_bwd_workspace_bytes(prob: Norm) -> int:
    return int(_load().ssd_bc_norm_bwd_workspace_bytes(ctypes.byref(prob)))


def bc_norm_bwd_into(prob: Norm, B, C, wB, wC, inv_freq, positions, dBn, dCn, dB, dC, dwB, dwC, ws,
                     stream=None) -> None:
    """Enqueue one backward into caller-provided gradients and workspace (no allocation)."""
    _call("ssd_bc_norm_bwd", prob, (B, C, wB, wC, inv_freq, positions, dBn, dCn, dB, dC, dwB, dwC), ws, stream)


def bc_norm_bwd(B, C, dBn, dCn, wB=None, wC=None, mode="rms", eps=1e-6, inv_freq=None, positions=None,
                interleaved=False, workspace=None):
    """Backward of bc_norm, given dBn and dCn (contiguous, like Bn and Cn).  Returns a dict with
    dB and dC (contiguous) and, for the weights that were given, dwB and dwC (float32 [N])."""
    import torch
    prob, need = _norm_problem(B, C, wB, wC, mode, eps, inv_freq, positions, interleaved)
    for name, t, like in (("dBn", dBn, B), ("dCn", dCn, C)):
        if t.shape != like.shape or t.dtype != like.dtype or t.get_device() != like.get_device() or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {like.dtype} tensor of shape {tuple(like.shape)} on {like.device}")
    out = dict(dB=torch.empty_like(dBn), dC=torch.empty_like(dCn))
    for name, w in (("dwB", wB), ("dwC", wC)):
        if w is not None:
            out[name] = torch.empty_like(w)
    ws = None
    if wB is not None or wC is not None:
        ws = _workspace(workspace, need, B.device)
    _call("ssd_bc_norm_bwd", prob, (B, C, wB, wC, inv_freq, positions, dBn, dCn, out["dB"], out["dC"], out.get("dwB"),
                                    out.get("dwC")), ws, index=B.get_device())
    return out
