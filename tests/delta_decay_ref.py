"""float64 reference of the gated delta rule's decay gradients with the sums of their absolute
terms, token by token from the definition."""
import torch


def decay_gradients(d, gr):
    """ddt, dA and s_t = sum over a state's elements of |g_t (I - beta_t B_t B_t^T)| |a_t h_{t-1}|, the
    absolute terms of ddt_t / A: the definition, float64, token by token."""
    f = {k: v.double() for k, v in {**d, **gr}.items() if v is not None}
    b, T, H, P = f["x"].shape
    rep = H // f["B"].shape[2]
    k, q = f["B"].repeat_interleave(rep, 2), f["C"].repeat_interleave(rep, 2)
    a = torch.exp(f["dt"] * f["A"])[..., None, None]
    outer = lambda p, n: p[..., None] * n[..., None, :]  # noqa: E731
    h, before = f["h0"], []
    for t in range(T):
        g = a[:, t] * h
        before.append(g)
        u = f["beta"][:, t, :, None] * (f["x"][:, t] - (g @ k[:, t, :, :, None])[..., 0])
        h = g + outer(u, k[:, t])
    lam = f["dhT"]
    D, s = torch.zeros(b, T, H, dtype=torch.float64), torch.zeros(b, T, H, dtype=torch.float64)
    for t in reversed(range(T)):
        lam = lam + outer(f["dy"][:, t], q[:, t])
        z = (lam @ k[:, t, :, :, None])[..., 0]
        lam = lam - outer(f["beta"][:, t, :, None] * z, k[:, t])
        D[:, t] = (lam * before[t]).sum((-1, -2))
        s[:, t] = (lam.abs() * before[t].abs()).sum((-1, -2))
        lam = lam * a[:, t]
    return D * f["A"], (D * f["dt"]).sum((0, 1)), s
