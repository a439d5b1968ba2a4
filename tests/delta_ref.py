"""float64 reference of the gated delta rule and of the norm of B and C, token by token from
the definitions (no chunks, no code shared with the library), and seeded inputs."""
import numpy as np
import torch


def make(b, T, H, P, N, G, seed, dtype="bf16", beta="sigmoid", dt_hi=0.1, key="unit", h0=True):
    """CPU tensors of one problem; x/B/C/beta already hold values of the problem dtype."""
    g = torch.Generator().manual_seed(seed)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda v: v / v.norm(dim=-1, keepdim=True)  # noqa: E731
    d = dict(x=rn(b, T, H, P).to(td), dt=torch.rand(b, T, H, generator=g) * dt_hi,
             A=-torch.exp(torch.rand(H, generator=g) * np.log(16.0)).float(),
             B=unit(rn(b, T, G, N)).to(td), C=unit(rn(b, T, G, N)).to(td),
             h0=0.1 * rn(b, H, P, N) if h0 else None)
    if key == "same":  # every token the same key: the strongest coupling inside a chunk
        d["B"] = d["B"][:, :1].expand(b, T, G, N).contiguous()
    if beta == "sigmoid":
        d["beta"] = torch.sigmoid(rn(b, T, H)).to(td)
    elif beta == "zeros":  # tokens that write nothing among others that do
        d["beta"] = (torch.sigmoid(rn(b, T, H)) * (torch.rand(b, T, H, generator=g) < 0.5)).to(td)
    else:
        d["beta"] = torch.full((b, T, H), float(beta)).to(td)
    return d


def make_grads(b, T, H, P, N, seed, dtype="bf16"):
    g = torch.Generator().manual_seed(seed + 77)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    return dict(dy=torch.randn(b, T, H, P, generator=g).to(td), dhT=0.1 * torch.randn(b, H, P, N, generator=g))


def residuals(d):
    """r of every token, float64 [b, T, H, P]."""
    out = []
    walk(d, keep=out)
    return torch.stack(out, 1)


def walk(d, h=None, weights=False, keep=None):
    """(y, hT) in float64, and with `weights` also the sums of absolute terms behind each y:
    what an error relative to every term of the sums is measured by."""
    f = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    x, dt, A, B, C, beta = (f[k] for k in ("x", "dt", "A", "B", "C", "beta"))
    b, T, H, P = x.shape
    rep, N = H // B.shape[2], B.shape[3]
    k, q = B.repeat_interleave(rep, 2), C.repeat_interleave(rep, 2)
    h = f["h0"] if h is None else h
    h = torch.zeros(b, H, P, N, dtype=torch.float64) if h is None else h
    mag, ys, yw = h.detach().abs(), [], []
    a = torch.exp(dt * A)
    for t in range(T):
        g = h * a[:, t, :, None, None]
        r = x[:, t] - (g @ k[:, t, :, :, None])[..., 0]
        if keep is not None:
            keep.append(r)
        u = beta[:, t, :, None] * r
        h = g + u[..., None] * k[:, t, :, None]
        ys.append((h @ q[:, t, :, :, None])[..., 0])
        if weights:
            mag = mag * a[:, t, :, None, None] + u.abs()[..., None] * k[:, t, :, None].abs()
            yw.append((mag @ q[:, t, :, :, None].abs())[..., 0])
    y = torch.stack(ys, 1) if T else x.clone()
    return (y, h, torch.stack(yw, 1) if T else x.clone()) if weights else (y, h)


GRAD_OF = dict(dx="x", ddt="dt", dA="A", dB="B", dC="C", dbeta="beta", dh0="h0")


def grads(d, gr):
    """Gradients of <dy, y> + <dhT, hT> by reverse-mode differentiation of the walk, float64."""
    f = {k: v.double().clone().requires_grad_() for k, v in d.items() if isinstance(v, torch.Tensor)}
    if d.get("h0") is None:
        b, T, H, P = d["x"].shape
        f["h0"] = torch.zeros(b, H, P, d["B"].shape[3], dtype=torch.float64, requires_grad=True)
    y, h = walk(f)
    loss = (y * gr["dy"].double()).sum()
    if gr.get("dhT") is not None:
        loss = loss + (h * gr["dhT"].double()).sum()
    names = list(GRAD_OF)
    got = torch.autograd.grad(loss, [f[GRAD_OF[n]] for n in names], allow_unused=True)
    return {n: (torch.zeros_like(f[GRAD_OF[n]]) if g is None else g) for n, g in zip(names, got)}


def norm(v, w, mode, eps, inv_freq, positions, interleaved):
    """One tensor [b, T, heads, N] in float64, differentiable."""
    v = v.double()
    s = v.square().sum(-1, keepdim=True) / (v.shape[-1] if mode == "rms" else 1)
    v = v / torch.sqrt(s + eps)
    if w is not None:
        v = v * w.double()
    if inv_freq is None:
        return v
    F = inv_freq.numel()
    ang = positions.double()[..., None, None] * inv_freq.double()
    i = torch.arange(F)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + F)
    a, b = v[..., lo], v[..., hi]
    out = v.clone()
    out[..., lo], out[..., hi] = a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()
    return out


def rel(got, ref):
    """||got - ref||_inf / ||ref||_inf over the whole tensor (0 for empty ones, inf for NaN)."""
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    if got.numel() == 0:
        return 0.0
    if not torch.isfinite(got).all():
        return float("inf")
    top = ref.abs().max().item()
    err = (got - ref).abs().max().item()
    return err / top if top > 0 else err
