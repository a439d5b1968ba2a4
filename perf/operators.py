"""Performance cases of the gated delta rule and of the norm of B and C.

Each case is one call of an operator at a size that it meets in use.  ``run`` makes the
call either through the package (``own``) or in a plain form written in elementary torch
operations; ``exact`` computes the same outputs in float64 from the definitions, token by
token.

The operators, for every batch row and head (B and C shared by the heads of a group):

    r_t = x_t - a_t h_{t-1} B_t,   h_t = a_t h_{t-1} + beta_t r_t B_t^T,   y_t = h_t C_t,
    a_t = exp(dt_t A)

(chunked forward, packed sequences, backward, and token by token on a held state), and the
norm of every row of B and C (rms or l2, optional weights) with the position rotation.
"""
import math

import torch

own = False

CHUNK = 64


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of one sequence: latency
        dict(name="step_one", op="step", b=1, T=1, H=32, P=128, N=128, G=16, dtype="bf16"),
        # one decode step of a served batch at the 2.7B layer's heads: bandwidth on the state
        dict(name="step_batch", op="step", b=64, T=1, H=80, P=64, N=128, G=1, dtype="bf16"),
        # a short prompt in float32, ragged last chunk: launch latency, the float32 path
        dict(name="fwd_small_f32", op="fwd", b=2, T=77, H=6, P=32, N=64, G=3, dtype="f32"),
        # training / prefill forward at the 2.7B layer shape, one group for all heads
        dict(name="fwd_layer", op="fwd", b=8, T=4096, H=80, P=64, N=128, G=1, dtype="bf16"),
        # one long sequence: few chains, many chunks, the widest state
        dict(name="fwd_long", op="fwd", b=1, T=65536, H=32, P=64, N=256, G=8, dtype="bf16"),
        # a served prefill batch of prompts of many lengths, packed
        dict(name="fwd_packed", op="packed", b=24, T=12001, H=32, P=128, N=128, G=16, dtype="bf16"),
        # a small training step in float32, ragged, shared heads
        dict(name="bwd_ragged_f32", op="bwd", b=2, T=333, H=4, P=64, N=64, G=2, dtype="f32"),
        # backward at the 780M layer shape
        dict(name="bwd_layer", op="bwd", b=2, T=2048, H=48, P=64, N=128, G=1, dtype="bf16"),
        # the norm and rotation before a decode step, far positions: latency
        dict(name="norm_decode", op="norm", b=32, T=1, GB=16, GC=16, N=128, F=32, mode="rms", weights=True,
             interleaved=False, far=1000000, dtype="bf16"),
        # the norm and rotation before a prefill or training forward
        dict(name="norm_layer", op="norm", b=8, T=4096, GB=16, GC=16, N=128, F=64, mode="rms", weights=True,
             interleaved=False, far=0, dtype="bf16"),
        # its backward, float32, odd token count, no rotation
        dict(name="norm_bwd_small_f32", op="norm_bwd", b=3, T=331, GB=2, GC=6, N=64, F=0, mode="l2", weights=False,
             interleaved=False, far=0, dtype="f32"),
        # its backward at the layer's size, weights' gradients over all tokens and heads
        dict(name="norm_bwd_layer", op="norm_bwd", b=8, T=4096, GB=16, GC=16, N=128, F=64, mode="rms", weights=True,
             interleaved=True, far=0, dtype="bf16"),
    ]


# what a drawn case may cost (bytes, flops), by operator: the listed ones' largest
_MOST = {"fwd": (740e6, 130e9), "packed": (740e6, 130e9), "bwd": (150e6, 55e9), "step": (350e6, 1e12),
         "norm": (540e6, 1e12), "norm_bwd": (810e6, 1e12)}


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "packed", "bwd", "bwd", "step", "norm", "norm_bwd"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op.startswith("norm"):
        N = rng.choice([16, 32, 64, 128, 256])
        c = dict(op=op, b=_log(rng, 1, 64), T=_log(rng, 1, 8192), GB=_log(rng, 1, 32), GC=_log(rng, 1, 32), N=N,
                 F=rng.choice([0, N // 4, N // 2, N // 2]), mode=rng.choice(["rms", "l2"]),
                 weights=rng.random() < 0.6, interleaved=rng.random() < 0.5, far=rng.choice([0, 0, 100000]),
                 dtype=dtype)
    else:
        G = rng.choice([1, 1, 2, 3, 4, 8])
        c = dict(op=op, b=_log(rng, 1, 32), T=_log(rng, 1, 16384), H=G * rng.choice([1, 2, 3, 4, 8]),
                 P=rng.choice([16, 32, 64, 64, 128]), N=rng.choice([16, 32, 64, 128, 128, 256]), G=G, dtype=dtype)
        if op == "step":
            c.update(b=_log(rng, 1, 256), T=rng.choice([1, 1, 1, 2, 5]))
    while True:
        w = work(c)
        scale = 4 if dtype == "f32" and op in ("fwd", "packed", "bwd") else 1  # the float32 path costs more
        if scale * w["bytes"] <= _MOST[op][0] and scale * w["flops"] <= _MOST[op][1]:
            return c
        big = "T" if c["T"] >= c["b"] else "b"
        c[big] = max(1, c[big] * 2 // 3)


def work(case):
    c, es = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"].startswith("norm"):
        rows = c["b"] * c["T"] * (c["GB"] + c["GC"])
        return dict(bytes=rows * c["N"] * es * (2 if c["op"] == "norm" else 3) + 4 * c["b"] * c["T"] * (c["F"] > 0),
                    flops=rows * c["N"] * 8)
    tok = c["T"] if c["op"] == "packed" else c["b"] * c["T"]
    x, bc, st = tok * c["H"] * c["P"] * es, tok * c["G"] * c["N"] * es, 4 * c["b"] * c["H"] * c["P"] * c["N"]
    gates, pn = tok * c["H"] * (4 + es), 2 * tok * c["H"] * c["P"] * c["N"]
    if c["op"] == "bwd":
        return dict(bytes=3 * x + 4 * bc + 2 * gates + 3 * st, flops=8 * pn)
    return dict(bytes=2 * x + 2 * bc + gates + 2 * st, flops=3 * pn)


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------
def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(int(seed))
    td = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    s = dict(case=dict(case))
    b, T, N = case["b"], case["T"], case["N"]
    if case["op"].startswith("norm"):
        # B and C are two slices of one projection's output
        GB, GC = case["GB"], case["GC"]
        proj = (normal(b, T, (GB + GC) * N) * 1.5 + 0.1).to(td)
        s["B"], s["C"] = proj[..., :GB * N].unflatten(-1, (GB, N)), proj[..., GB * N:].unflatten(-1, (GC, N))
        s["wB"], s["wC"] = ((1 + 0.1 * normal(N), 1 + 0.1 * normal(N)) if case["weights"] else (None, None))
        F = case["F"]
        s["inv_freq"] = (10000.0 ** (-torch.arange(F, device=dev, dtype=torch.float64) / F)).float() if F else None
        start = (uniform(b, 1) * case["far"]).to(torch.int32)
        s["positions"] = (torch.arange(T, device=dev, dtype=torch.int32)[None] + start).contiguous() if F else None
        if case["op"] == "norm_bwd":
            s["dBn"], s["dCn"] = normal(b, T, GB, N).to(td), normal(b, T, GC, N).to(td)
        return s
    H, P, G = case["H"], case["P"], case["G"]
    lead, rows = ((T,), b) if case["op"] == "packed" else ((b, T), b)

    def unit(v):
        return v / v.norm(dim=-1, keepdim=True)

    s["x"] = normal(*lead, H, P).to(td)
    # per head step sizes between 1e-3 and 0.1, decays exp(dt A) with A in [-16, -1]
    d = torch.exp(uniform(H) * math.log(100.0) + math.log(1e-3))
    bias = d + torch.log(-torch.expm1(-d))
    s["dt"] = torch.nn.functional.softplus(0.5 * normal(*lead, H) + bias).clamp(1e-3, 0.1).contiguous()
    s["A"] = -torch.exp(uniform(H) * math.log(16.0))
    s["B"], s["C"] = unit(normal(*lead, G, N)).to(td), unit(normal(*lead, G, N)).to(td)
    s["beta"] = torch.sigmoid(normal(*lead, H)).to(td)
    s["h0"] = 0.1 * normal(rows, H, P, N)
    if case["op"] == "step":
        s["h"] = s.pop("h0")
    if case["op"] == "bwd":
        s["dy"], s["dhT"] = normal(b, T, H, P).to(td), 0.1 * normal(b, H, P, N)
    if case["op"] == "packed":
        # lengths as uneven as prompts are; the last ones may be empty
        share = torch.exp(1.2 * normal(b).double())
        cu = torch.cat([torch.zeros(1, device=dev, dtype=torch.float64), share.cumsum(0) / share.sum()]) * T
        s["cu_seqlens"] = cu.round().to(torch.int32)
    return s


# --------------------------------------------------------------------------------------
# the calls
# --------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        import ssd_chunked_scan_03_amd as ssd
        if c["op"] == "fwd":
            return ssd.delta_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["beta"], s["h0"])
        if c["op"] == "packed":
            return ssd.delta_fwd_varlen(s["x"], s["dt"], s["A"], s["B"], s["C"], s["beta"], s["cu_seqlens"], s["h0"])
        if c["op"] == "bwd":
            return ssd.delta_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["beta"], s["dy"], s["h0"], s["dhT"])
        if c["op"] == "step":
            return ssd.delta_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["beta"], s["h"]), s["h"]
        kw = dict(mode=c["mode"], eps=1e-6, inv_freq=s["inv_freq"], positions=s["positions"],
                  interleaved=c["interleaved"])
        if c["op"] == "norm":
            return ssd.bc_norm(s["B"], s["C"], s["wB"], s["wC"], **kw)
        return ssd.bc_norm_bwd(s["B"], s["C"], s["dBn"], s["dCn"], s["wB"], s["wC"], **kw)
    return _PLAIN[c["op"]](s)


# --------------------------------------------------------------------------------------
# plain forms (float32 products, float64 decay sums, rounded once)
# --------------------------------------------------------------------------------------
def _by_chunk(v, heads):
    """[b, T, heads' groups, n] (or [b, T, H]) -> [b, H, chunks, CHUNK, n] float32, zeros past T."""
    v = v.float()
    v = v.unsqueeze(-1) if v.dim() == 3 else v
    b, T, g, n = v.shape
    nc = max(1, -(-T // CHUNK))
    out = v.new_zeros(b, nc * CHUNK, g, n)
    out[:, :T] = v
    out = out.permute(0, 2, 1, 3).reshape(b, g, nc, CHUNK, n)
    return out if g == heads else out.repeat_interleave(heads // g, dim=1)


def _inverse(low):
    """(I + low)^-1 for strictly lower `low`, by doubling the size of the inverted diagonal blocks."""
    n = low.shape[-1]
    i = torch.arange(n, device=low.device)
    inv = torch.eye(n, device=low.device, dtype=low.dtype).expand(low.shape).contiguous()
    size = 1
    while size < n:
        same, left = i[:, None] // (2 * size) == i[None] // (2 * size), (i // size) % 2
        inv = inv - inv @ (low * (same & (left[:, None] == 1) & (left[None] == 0))) @ inv
        size *= 2
    return inv


def _tables(s):
    H = s["x"].shape[2]
    t = dict(q=_by_chunk(s["C"], H), k=_by_chunk(s["B"], H), v=_by_chunk(s["x"], H), beta=_by_chunk(s["beta"], H))
    dt = _by_chunk(s["dt"], H)
    cum = (dt.double() * s["A"].double()[None, :, None, None, None]).cumsum(-2)
    t["dt"], t["ec"], t["ew"] = dt, cum.exp().float(), (cum[..., -1:, :] - cum).exp().float()
    t["el"] = cum[..., -1:, :].exp().float()
    t["gam"] = (cum - cum.transpose(-1, -2)).clamp(max=0).exp().float().tril()
    kt = t["k"].transpose(-1, -2)
    t["kk"], t["m"] = (t["k"] @ kt * t["gam"]).tril(-1), t["q"] @ kt * t["gam"]
    t["inv"] = _inverse(t["beta"] * t["kk"])
    return t


def _states(t, h):
    """The state entering every chunk, every chunk's u, and the last state."""
    u0, w = t["inv"] @ (t["beta"] * t["v"]), t["inv"] @ (t["beta"] * t["ec"] * t["k"])
    hs, us = [], []
    for c in range(t["k"].shape[2]):
        hs.append(h)
        us.append(u0[:, :, c] - w[:, :, c] @ h.transpose(-1, -2))
        h = t["el"][:, :, c] * h + (t["ew"][:, :, c] * us[-1]).transpose(-1, -2) @ t["k"][:, :, c]
    return torch.stack(hs, 2), torch.stack(us, 2), h


def _tokens(v, T, dtype):
    """[b, H, chunks, CHUNK, n] -> [b, T, H, n]."""
    b, H, nc, L, n = v.shape
    return v.reshape(b, H, nc * L, n)[:, :, :T].permute(0, 2, 1, 3).to(dtype).contiguous()


def _plain_fwd(s):
    t = _tables(s)
    hs, us, hT = _states(t, s["h0"])
    y = t["ec"] * (t["q"] @ hs.transpose(-1, -2)) + t["m"] @ us
    return _tokens(y, s["x"].shape[1], s["x"].dtype), hT


def _plain_packed(s):
    cu = s["cu_seqlens"].long()
    T, n = s["x"].shape[0], cu.numel() - 1
    lens = cu[1:] - cu[:-1]
    most = int(lens.max())
    tok = torch.arange(T, device=cu.device)
    row = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    pos = tok - cu[row]
    p = dict(A=s["A"], h0=s["h0"])
    for k in ("x", "dt", "B", "C", "beta"):
        p[k] = s[k].new_zeros(n, most, *s[k].shape[1:])
        p[k][row, pos] = s[k]
    y, hT = _plain_fwd(p)
    return y[row, pos], hT


def _plain_bwd(s):
    t = _tables(s)
    b, T, H, P = s["x"].shape
    G = s["B"].shape[2]
    hs, us, hT = _states(t, s["h0"])
    dy = _by_chunk(s["dy"], H)
    du0, lam, lams, zs = t["m"].transpose(-1, -2) @ dy, s["dhT"], [], []
    for c in reversed(range(dy.shape[2])):
        k = t["k"][:, :, c]
        lams.append(lam)
        zs.append(t["inv"][:, :, c].transpose(-1, -2) @ (du0[:, :, c] + t["ew"][:, :, c] * (k @ lam.transpose(-1, -2))))
        lam = (t["el"][:, :, c] * lam + (t["ec"][:, :, c] * dy[:, :, c]).transpose(-1, -2) @ t["q"][:, :, c]
               - (t["ec"][:, :, c] * t["beta"][:, :, c] * zs[-1]).transpose(-1, -2) @ k)
    lams, z = torch.stack(lams[::-1], 2), torch.stack(zs[::-1], 2)
    dx = t["beta"] * z
    r = t["v"] - t["ec"] * (t["k"] @ hs.transpose(-1, -2)) - t["kk"] @ us
    y = t["ec"] * (t["q"] @ hs.transpose(-1, -2)) + t["m"] @ us
    dp = (dy @ us.transpose(-1, -2)) * t["gam"]
    dg = -(t["beta"] * (z @ us.transpose(-1, -2)) * t["gam"]).tril(-1)
    dq = t["ec"] * (dy @ hs) + dp @ t["k"]
    dk = (dp.transpose(-1, -2) @ t["q"] + dg @ t["k"] + dg.transpose(-1, -2) @ t["k"] + t["ew"] * (us @ lams)
          - t["ec"] * (dx @ hs))
    after = torch.cat([hs[:, :, 1:], hT[:, :, None]], 2)
    terms = (dy * y).double().sum(-1, keepdim=True) - (dx * t["v"]).double().sum(-1, keepdim=True)
    dlog = terms.flip(-2).cumsum(-2).flip(-2) + (lams * after).double().sum((-1, -2), keepdim=True)
    shared = lambda v: v.unflatten(1, (G, H // G)).sum(2)  # noqa: E731
    td = s["x"].dtype
    return dict(dx=_tokens(dx, T, td), ddt=_tokens(dlog * s["A"].double()[None, :, None, None, None], T, torch.float32)[..., 0].contiguous(),
                dA=(t["dt"] * dlog).sum((0, 2, 3, 4)).float(), dB=_tokens(shared(dk), T, td),
                dC=_tokens(shared(dq), T, td), dbeta=_tokens((z * r).sum(-1, keepdim=True), T, td)[..., 0].contiguous(),
                dh0=lam)


def _plain_step(s):
    h, H = s["h"], s["x"].shape[2]
    rep = H // s["B"].shape[2]
    k, q = s["B"].float().repeat_interleave(rep, 2), s["C"].float().repeat_interleave(rep, 2)
    x, beta, a = s["x"].float(), s["beta"].float(), (s["dt"] * s["A"]).exp()
    ys = []
    for t in range(x.shape[1]):
        g = h * a[:, t, :, None, None]
        r = x[:, t] - (g * k[:, t, :, None]).sum(-1)
        h = g + (beta[:, t, :, None] * r)[..., None] * k[:, t, :, None]
        ys.append((h * q[:, t, :, None]).sum(-1))
    s["h"].copy_(h)
    return torch.stack(ys, 1).to(s["x"].dtype), s["h"]


def _angles(s):
    turn = s["positions"].double()[..., None] * s["inv_freq"].double()
    return turn.cos().float()[:, :, None], turn.sin().float()[:, :, None]


def _halves(c, v):
    F = c["F"]
    return (v[..., 0:2 * F:2], v[..., 1:2 * F:2]) if c["interleaved"] else (v[..., :F], v[..., F:2 * F])


def _turned(c, v, cos, sin):
    p, q = _halves(c, v)
    a, b = p * cos - q * sin, p * sin + q * cos
    both = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([both, v[..., 2 * c["F"]:]], -1)


def _plain_norm(s):
    c = s["case"]
    cs = _angles(s) if c["F"] else None

    def one(v, w):
        x = v.float()
        sq = (x * x).sum(-1, keepdim=True) * (1.0 / c["N"] if c["mode"] == "rms" else 1.0)
        x = x * torch.rsqrt(sq + 1e-6)
        x = x if w is None else x * w
        return (_turned(c, x, *cs) if cs else x).to(v.dtype).contiguous()

    return one(s["B"], s["wB"]), one(s["C"], s["wC"])


def _plain_norm_bwd(s):
    c = s["case"]
    cs = _angles(s) if c["F"] else None
    scale = 1.0 / c["N"] if c["mode"] == "rms" else 1.0

    def one(v, w, dv):
        x, g = v.float(), dv.float()
        g = _turned(c, g, cs[0], -cs[1]) if cs else g
        r = torch.rsqrt((x * x).sum(-1, keepdim=True) * scale + 1e-6)
        dw = None if w is None else (g * x * r).double().sum((0, 1, 2)).float()
        g = g if w is None else g * w
        return (r * g - scale * r * r * r * x * (x * g).sum(-1, keepdim=True)).to(v.dtype).contiguous(), dw

    (dB, dwB), (dC, dwC) = one(s["B"], s["wB"], s["dBn"]), one(s["C"], s["wC"], s["dCn"])
    out = dict(dB=dB, dC=dC)
    return out if dwB is None else dict(out, dwB=dwB, dwC=dwC)


_PLAIN = dict(fwd=_plain_fwd, packed=_plain_packed, bwd=_plain_bwd, step=_plain_step, norm=_plain_norm,
              norm_bwd=_plain_norm_bwd)


# --------------------------------------------------------------------------------------
# float64 values from the definitions, token by token
# --------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    if case["op"] == "packed":
        return _exact_packed(s)
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if case["op"] == "bwd":
        return _exact_bwd(f)
    y, h = _walk(f, f["h"] if case["op"] == "step" else f["h0"])
    return torch.stack(y, 1), h


def _walk(f, h, keep=None):
    """The recurrence over [b, T] tokens; `keep` collects (state before, decayed state, r) of every token."""
    rep = f["x"].shape[2] // f["B"].shape[2]
    k, q = f["B"].repeat_interleave(rep, 2), f["C"].repeat_interleave(rep, 2)
    a = torch.exp(f["dt"] * f["A"])
    ys = []
    for t in range(f["x"].shape[1]):
        g = h * a[:, t, :, None, None]
        r = f["x"][:, t] - torch.einsum("bhpn,bhn->bhp", g, k[:, t])
        h = g + torch.einsum("bhp,bhn->bhpn", f["beta"][:, t, :, None] * r, k[:, t])
        ys.append(torch.einsum("bhpn,bhn->bhp", h, q[:, t]))
        if keep is not None:
            keep.append((g, h, r))
    return ys, h


def _exact_packed(s):
    ends = s["cu_seqlens"].tolist()
    ys, hs = [], []
    order = sorted(range(len(ends) - 1), key=lambda i: ends[i + 1] - ends[i])
    most = max(ends[i + 1] - ends[i] for i in order)
    if most * 12 > 1500000:
        return None
    # every sequence padded to the longest: a token with beta = 0 and dt = 0 leaves the state
    n = len(order)
    f = dict(A=s["A"].double())
    for key in ("x", "dt", "B", "C", "beta"):
        f[key] = torch.zeros(n, most, *s[key].shape[1:], device=s[key].device, dtype=torch.float64)
        for i in range(n):
            f[key][i, :ends[i + 1] - ends[i]] = s[key][ends[i]:ends[i + 1]].double()
    y, h = _walk(f, s["h0"].double())
    y = torch.stack(y, 1)
    return torch.cat([y[i, :ends[i + 1] - ends[i]] for i in range(n)]), h


def _exact_bwd(f, span=64):
    b, T, H, P = f["x"].shape
    G, N = f["B"].shape[2:]
    rep = H // G
    k, q = f["B"].repeat_interleave(rep, 2), f["C"].repeat_interleave(rep, 2)
    a = torch.exp(f["dt"] * f["A"])
    part = lambda i: {n: (v[:, i:i + span] if n in ("x", "dt", "B", "C", "beta") else v) for n, v in f.items()}  # noqa: E731
    starts, h = [], f["h0"]
    for i in range(0, T, span):
        starts.append(h)
        _, h = _walk(part(i), h)
    lam = f["dhT"]
    dx, dlog, dbeta = torch.zeros_like(f["x"]), torch.zeros_like(f["dt"]), torch.zeros_like(f["dt"])
    dk, dq = torch.zeros_like(k), torch.zeros_like(q)
    for i in reversed(range(0, T, span)):
        kept = []
        _walk(part(i), starts[i // span], kept)
        for t in reversed(range(i, min(T, i + span))):
            g, ht, r = kept[t - i]
            lam = lam + torch.einsum("bhp,bhn->bhpn", f["dy"][:, t], q[:, t])
            dq[:, t] = torch.einsum("bhpn,bhp->bhn", ht, f["dy"][:, t])
            z = torch.einsum("bhpn,bhn->bhp", lam, k[:, t])
            bt = f["beta"][:, t, :, None]
            dbeta[:, t], dx[:, t] = (z * r).sum(-1), bt * z
            dk[:, t] = bt * torch.einsum("bhpn,bhp->bhn", lam, r) - torch.einsum("bhpn,bhp->bhn", g, bt * z)
            lam = lam - torch.einsum("bhp,bhn->bhpn", bt * z, k[:, t])
            dlog[:, t] = (lam * g).sum((-1, -2))
            lam = lam * a[:, t, :, None, None]
    shared = lambda v: v.unflatten(2, (G, rep)).sum(3)  # noqa: E731
    return dict(dx=dx, ddt=dlog * f["A"], dA=(dlog * f["dt"]).sum((0, 1)), dB=shared(dk), dC=shared(dq), dbeta=dbeta,
                dh0=lam)


def _exact_norm(s):
    c, out = s["case"], []
    F, N = c["F"], c["N"]
    for v, w, dv in ((s["B"], s["wB"], s.get("dBn")), (s["C"], s["wC"], s.get("dCn"))):
        x = v.double()
        n = (x.square().mean(-1, keepdim=True) if c["mode"] == "rms" else x.square().sum(-1, keepdim=True)) + 1e-6
        hat = x / n.sqrt()
        gain = torch.ones(N, device=x.device, dtype=torch.float64) if w is None else w.double()
        turn = (torch.polar(torch.ones(()).double().to(x.device), s["positions"].double()[..., None, None] * s["inv_freq"].double())
                if F else None)

        def rotate(u, by):
            if not F:
                return u
            i = torch.arange(F, device=u.device)
            lo, hi = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + F)
            z = torch.complex(u[..., lo], u[..., hi]) * by
            u = u.clone()
            u[..., lo], u[..., hi] = z.real, z.imag
            return u

        if dv is None:
            out.append(rotate(hat * gain, turn))
            continue
        g = rotate(dv.double(), turn.conj() if F else None)
        dw = (g * hat).sum((0, 1, 2))
        g = g * gain
        out.append(((g - hat * (g * hat).sum(-1, keepdim=True) / (N if c["mode"] == "rms" else 1)) / n.sqrt(), dw))
    if c["op"] == "norm":
        return tuple(out)
    d = dict(dB=out[0][0], dC=out[1][0])
    return dict(d, dwB=out[0][1], dwC=out[1][1]) if c["weights"] else d
