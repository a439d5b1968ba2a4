"""GPU parity of the norm and rotation of B and C with its float64 definition.

Tolerances.  A row's result is rounded once: 2^-8 (bfloat16) of the value; behind it float32
arithmetic: the sum of up to 256 squares by 8 in a lane and then pairs (13 steps), the
root, the scale, the cosine and the turn, about 24 roundings of 2^-24 relative to the pair's
length, which a turn may leave much larger than one of its two values: 24 2^-24 of the row's
largest value.  The backward has twice as many steps, and its row sum takes the largest of
|g x| N / N.  The weights' gradients sum up to 10^3 rows in float32 per work-group: 2e-5 of
the sum of absolute terms.
"""
import pytest
import torch

import delta_ref as ref
import ssd_chunked_scan_03_amd as ssd

pytestmark = pytest.mark.gpu
B16, F32 = 2.0 ** -8, 2.0 ** -24


def problem(b, T, GB, GC, N, F, dtype, seed, weights=True, far=0, strided=True):
    g = torch.Generator().manual_seed(seed)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    pad = 16
    proj = (torch.randn(b, T, (GB + GC) * N + pad, generator=g) * 2).to(td)
    d = dict(proj=proj, wB=1 + torch.randn(N, generator=g) if weights else None,
             wC=1 + torch.randn(N, generator=g) if weights else None,
             inv_freq=(10000.0 ** (-torch.arange(F).double() / F)).float() if F else None,
             positions=(torch.arange(T)[None] + torch.randint(0, far + 1, (b, 1), generator=g)).to(torch.int32) if F else None,
             dBn=torch.randn(b, T, GB, N, generator=g).to(td), dCn=torch.randn(b, T, GC, N, generator=g).to(td))
    return d


def views(proj, GB, GC, N):
    return proj[..., :GB * N].unflatten(-1, (GB, N)), proj[..., GB * N:(GB + GC) * N].unflatten(-1, (GC, N))


def cuda(v):
    return v if v is None else v.cuda()


def close(got, want, dtype, steps, where):
    got, want = got.double().cpu(), want.detach().double()
    assert got.shape == want.shape and torch.isfinite(got).all(), where
    if not got.numel():
        return
    lim = (B16 if dtype == "bf16" else F32) * want.abs() + steps * F32 * want.abs().amax(-1, keepdim=True)
    worst = ((got - want).abs() / lim.clamp(min=1e-30)).max().item()
    assert worst <= 1.0, (where, worst)


# b, T, GB, GC, N, F, dtype, mode, interleaved, weights, far
CASES = [
    (1, 1, 1, 1, 16, 0, "bf16", "rms", False, True, 0),
    (1, 1, 1, 2, 16, 4, "f32", "l2", False, False, 10),       # 4 elements per lane
    (2, 3, 2, 1, 32, 16, "bf16", "l2", False, True, 0),
    (2, 5, 3, 5, 64, 12, "f32", "rms", False, True, 100),     # partial rotation, 4 per lane
    (3, 7, 1, 6, 128, 64, "bf16", "rms", True, True, 5),
    (1, 9, 4, 4, 256, 128, "f32", "l2", False, True, 0),
    (2, 4, 2, 2, 256, 100, "bf16", "rms", False, False, 7),
    (1, 3, 2, 2, 128, 60, "f32", "rms", True, False, 2000000000),  # far positions
    (1, 2, 0, 3, 64, 32, "bf16", "rms", False, True, 0),      # one tensor without heads
    (2, 2100, 1, 1, 16, 8, "bf16", "rms", False, True, 0),    # four tokens per work-group, ragged
]
IDS = ["-".join(map(str, c)) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_norm_matches_definition(case):
    b, T, GB, GC, N, F, dtype, mode, il, weights, far = case
    print(f"[bc_norm] {case}", flush=True)
    d = problem(b, T, GB, GC, N, F, dtype, 31, weights, far)
    B, C = views(d["proj"].cuda(), GB, GC, N)
    Bn, Cn = ssd.bc_norm(B, C, cuda(d["wB"]), cuda(d["wC"]), mode=mode, eps=1e-5, inv_freq=cuda(d["inv_freq"]),
                         positions=cuda(d["positions"]), interleaved=il)
    for got, v, w in zip((Bn, Cn), views(d["proj"], GB, GC, N), (d["wB"], d["wC"])):
        close(got, ref.norm(v, w, mode, 1e-5, d["inv_freq"], d["positions"], il), dtype, 24, case)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_norm_backward_matches_reverse_mode(case):
    b, T, GB, GC, N, F, dtype, mode, il, weights, far = case
    print(f"[bc_norm backward] {case}", flush=True)
    d = problem(b, T, GB, GC, N, F, dtype, 32, weights, far)
    B, C = views(d["proj"].cuda(), GB, GC, N)
    out = ssd.bc_norm_bwd(B, C, d["dBn"].cuda(), d["dCn"].cuda(), cuda(d["wB"]), cuda(d["wC"]), mode=mode, eps=1e-5,
                          inv_freq=cuda(d["inv_freq"]), positions=cuda(d["positions"]), interleaved=il)
    assert set(out) == ({"dB", "dC", "dwB", "dwC"} if weights else {"dB", "dC"})
    for n, wn, dv, v, w in (("dB", "dwB", d["dBn"], views(d["proj"], GB, GC, N)[0], d["wB"]),
                            ("dC", "dwC", d["dCn"], views(d["proj"], GB, GC, N)[1], d["wC"])):
        f = v.double().clone().requires_grad_()
        gw = None if w is None else w.double().clone().requires_grad_()
        y = ref.norm(f, gw, mode, 1e-5, d["inv_freq"], d["positions"], il)
        grads = torch.autograd.grad((y * dv.double()).sum(), [f] if gw is None else [f, gw])
        # a sum over the row of terms up to |g x| each, times |x|: relative to the row's largest
        # gradient before the projection takes a part of it away
        r = 1 / torch.sqrt(f.square().sum(-1, keepdim=True) / (N if mode == "rms" else 1) + 1e-5)
        top = (r * dv.double().abs().amax(-1, keepdim=True) * (1 if w is None else w.double().abs().max()) * 2).detach()
        got = out[n].double().cpu()
        lim = (B16 if dtype == "bf16" else F32) * grads[0].abs() + 48 * F32 * (grads[0].abs() + top)
        assert torch.isfinite(got).all()
        if got.numel():
            assert ((got - grads[0]).abs() / lim).max().item() <= 1.0, case
        if gw is not None and GB * GC:
            terms = (dv.double().abs() * 2 * (f.detach() * r.detach()).abs().amax(-1, keepdim=True)).sum((0, 1, 2))
            assert ((out[wn].double().cpu() - grads[1]).abs() / (2e-5 * terms + 1e-30)).max().item() <= 1.0, case


def test_zero_and_large_rows():
    """A zero row stays zero (eps keeps its root), its gradient finite; rows of 1e18 do not
    overflow: their squares reach 1e36 and 256 of them 3e38 stays under float32's largest."""
    x = torch.zeros(1, 3, 1, 64, device="cuda")
    x[0, 1] = 1e18
    x[0, 2] = 1e-20
    Bn, Cn = ssd.bc_norm(x, x, mode="rms")
    assert (Bn[0, 0] == 0).all() and torch.isfinite(Bn).all()
    assert torch.allclose(Bn[0, 1], torch.ones(1, 64, device="cuda"), rtol=1e-6)
    out = ssd.bc_norm_bwd(x, x, torch.ones_like(x), torch.ones_like(x), mode="rms")
    assert torch.isfinite(out["dB"]).all()


def test_default_positions_and_determinism():
    d = problem(2, 50, 2, 2, 64, 32, "bf16", 33)
    B, C = (v.contiguous().cuda() for v in views(d["proj"], 2, 2, 64))
    pos = torch.arange(50, dtype=torch.int32, device="cuda").expand(2, 50).contiguous()
    freq = d["inv_freq"].cuda()
    a = ssd.bc_norm(B, C, inv_freq=freq)
    b = ssd.bc_norm(B, C, inv_freq=freq, positions=pos)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    args = (B, C, d["dBn"].cuda(), d["dCn"].cuda(), d["wB"].cuda(), d["wC"].cuda())
    g0, g1 = ssd.bc_norm_bwd(*args), ssd.bc_norm_bwd(*args)
    assert all(torch.equal(g0[k], g1[k]) for k in g0)


def test_no_tokens():
    B = torch.zeros(2, 0, 2, 32, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(32, device="cuda")
    assert ssd.bc_norm(B, B, w, w)[0].shape == B.shape
    out = ssd.bc_norm_bwd(B, B, B, B, w, w)
    assert (out["dwB"] == 0).all() and (out["dwC"] == 0).all()


def test_normed_inputs_of_the_scan():
    """bc_norm before the scan: the scan of the normed B and C, against the scan's definition."""
    import numpy as np
    import oracle
    from helpers import rel_h, rel_y
    from ssd_chunked_scan_03_amd.synth import make_small
    inp = make_small(2, 130, 4, 64, 64, 2, seed=35, dtype="f32")
    t = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in inp.items() if v is not None and "bits" not in k}
    freq = (100.0 ** (-torch.arange(32) / 32)).float().cuda()
    Bn, Cn = ssd.bc_norm(t["B"], t["C"], mode="l2", inv_freq=freq)
    y, hT = ssd.scan_fwd(t["x"], t["dt"], t["A"], Bn, Cn, t["D"], t["h0"], chunk=64)
    pos = torch.arange(130).expand(2, 130)
    nb, nc = (ref.norm(torch.from_numpy(inp[k]), None, "l2", 1e-6, freq.cpu(), pos, False).numpy() for k in ("B", "C"))
    yr, hr = oracle.recurrence(inp["x"], inp["dt"], inp["A"], nb, nc, inp["D"], inp["h0"], diag=False)
    assert rel_y(y.cpu().numpy(), yr) < 1e-4 and rel_h(hT.cpu().numpy(), hr) < 1e-4
