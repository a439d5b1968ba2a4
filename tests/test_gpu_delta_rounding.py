"""The bfloat16 results of the gated delta rule against their own rounding: what each is off by
beside it, in the mean square over the whole tensor.

y: as test_gpu_delta derives it, at shapes that run two column tiles a team, and a wave per 16
columns at dstate 256.

Gradients.  With values rounded to bfloat16 independently, the squares of their errors add.  A
rounding's mean square is (2^-7)^2 / 12 of the power of two below the value, so RHO = 2^-14 / 12 of
the value's square at most; two terms leave 2^-18 of a value.
* dx = beta z is rounded once.
* dbeta = z . r, r and z in two terms, their smallest product left out: 3 2^-18 of sum_p |z_p r_p|.
* dC = e^c dY h + dP K: the entering state h in one term, so RHO of the sum of squares of its
  products; r in two terms and dP in two: 2 2^-18 of G_ij sum_p |dY_i u_j| |K_j|.
* dB = dP^T Q + (W + W^T) K + e^{c_L - c} u dh' - e^c dX h: likewise h and the leaving adjoint dh', and
  the two tables (z too: 4 2^-18).
float32 sums behind all of it: F32 of the absolute terms where they are named, far below the rest.
"""
import pytest
import torch

import delta_ref as ref
import test_gpu_delta as base

pytestmark = pytest.mark.gpu
RHO, TWO = 2.0 ** -14 / 12, 2.0 ** -18
L = 64


@pytest.mark.parametrize("case", [(1, 130, 80, 64, 128, 8), (1, 70, 40, 128, 64, 2), (1, 130, 160, 64, 256, 8)],
                         ids=lambda c: "b{}T{}H{}P{}N{}G{}".format(*c))
@pytest.mark.parametrize("key", ["unit", "same"])
def test_y_of_other_walks(case, key):
    base.test_y_is_good_to_its_own_rounding(case, key)


def walks(d, gr):
    """float64: r and z of every token, the state entering and the adjoint leaving every chunk."""
    f = {k: v.double() for k, v in {**d, **gr}.items() if v is not None}
    T, H = f["x"].shape[1:3]
    rep = H // f["B"].shape[2]
    k, q = f["B"].repeat_interleave(rep, 2), f["C"].repeat_interleave(rep, 2)
    a = torch.exp(f["dt"] * f["A"])[..., None, None]
    outer = lambda p, n: p[..., None] * n[..., None, :]  # noqa: E731
    h, hin, rs = f["h0"], [], []
    for t in range(T):
        if t % L == 0:
            hin.append(h)
        g = a[:, t] * h
        rs.append(f["x"][:, t] - (g @ k[:, t, :, :, None])[..., 0])
        h = g + outer(f["beta"][:, t, :, None] * rs[-1], k[:, t])
    lam, lout, zs = f["dhT"], [], []
    for t in reversed(range(T)):
        if t % L == L - 1 or t == T - 1:
            lout.append(lam)
        lam = lam + outer(f["dy"][:, t], q[:, t])
        zs.append((lam @ k[:, t, :, :, None])[..., 0])
        lam = (lam - outer(f["beta"][:, t, :, None] * zs[-1], k[:, t])) * a[:, t]
    return f, k, q, torch.stack(rs, 1), torch.stack(zs[::-1], 1), hin, lout[::-1]


def beside_rounding(d, gr):
    """Mean squares that each gradient may be off by beside its own rounding, summed over the
    tensor."""
    f, K, Q, r, z, hin, lout = walks(d, gr)
    T, H = f["x"].shape[1:3]
    beta = f["beta"][..., None]
    u, dx = beta * r, beta * z
    sq = dict(dx=0.0, dbeta=((3 * TWO + base.F32) * (z * r).abs().sum(-1)).square().sum(), dB=0.0, dC=0.0)
    heads = lambda v: v.transpose(1, 2)  # [b, T, H, n] -> [b, H, T, n]  # noqa: E731
    for c, t0 in enumerate(range(0, T, L)):
        s = slice(t0, min(T, t0 + L))
        cum = (f["dt"][:, s] * f["A"]).cumsum(1).transpose(1, 2)  # [b, H, t]
        ec, ew = cum.exp()[..., None], (cum[..., -1:] - cum).exp()[..., None]
        gam = (cum[..., :, None] - cum[..., None, :]).clamp(max=0).exp().tril()
        dY, U, Z, X = (heads(v[:, s]) for v in (f["dy"], u, z, dx))
        k2, q2 = heads(K[:, s]).square(), heads(Q[:, s]).square()
        pq = (2 * TWO * gam * (dY.abs() @ U.abs().transpose(-1, -2))).square()          # of dP_ij
        pw = (4 * TWO * gam.tril(-1) * (X.abs() @ U.abs().transpose(-1, -2))).square()  # of W_ij
        h2, l2 = hin[c].square(), lout[c].square()
        sq["dC"] += (RHO * ((ec * dY).square() @ h2) + pq @ k2).sum()
        sq["dB"] += (RHO * ((ew * U).square() @ l2 + (ec * X).square() @ h2) + pq.transpose(-1, -2) @ q2
                     + (pw + pw.transpose(-1, -2)) @ k2).sum()
    return sq


@pytest.mark.parametrize("case", [(2, 130, 4, 64, 64, 2), (1, 130, 8, 64, 128, 2), (1, 100, 4, 128, 256, 1), (2, 130, 4, 32, 32, 2),
                                  (1, 130, 80, 64, 128, 8)], ids=lambda c: "b{}T{}H{}P{}N{}G{}".format(*c))
@pytest.mark.parametrize("dt_hi", [0.02, 0.2])
def test_gradients_are_good_to_their_roundings(case, dt_hi):
    """Each gradient's mean square error against its own rounding's and what its factors' leave, with 5%
    for the spread of so many roundings."""
    b, T, H, P, N, G = case
    print(f"[delta gradients' roundings] {case} {dt_hi}", flush=True)
    d, gr = ref.make(b, T, H, P, N, G, 56, "bf16", dt_hi=dt_hi), ref.make_grads(b, T, H, P, N, 56, "bf16")
    out, want, beside = base.backward(d, gr), ref.grads(d, gr), beside_rounding(d, gr)
    worst = {}
    for n, more in beside.items():
        own = (want[n].to(torch.bfloat16).double() - want[n]).square().sum()
        worst[n] = ((out[n].double().cpu() - want[n]).square().sum() / (own + more)).item()
    assert all(v < 1.05 for v in worst.values()), (case, worst)
    print(worst)
