"""GPU parity of the gated delta rule (chunked, packed, token by token, backward) with the
float64 walk of its definition.

Tolerances.  A bfloat16 rounding is off by at most 2^-8 of the value, a float32 one by 2^-24.
* y: the output is rounded once and the chunk's table M once, so with w_t = |C_t| . |h|_t the
  sum of the absolute terms behind y, |error| <= 2^-8 |y| + 2^-8 w (bfloat16).
* float32 results (hT, ddt, dA, dh0, and everything of a float32 problem): sums of dstate
  products, of a chunk's 64 tokens and of the chunks, each step off by 2^-24 of terms that
  the largest value of the result bounds up to their number: (256 + 64 + 64) 2^-24 = 2.3e-5
  of the largest value.
* gradients in bfloat16, relative to the largest value: dx is rounded once; dC is rounded and
  one factor of each of its products is (the state, or r): 2; dB's products have two rounded
  factors (r and dh', z and h): 3.  Each times 2^-8.  dbeta = sum_p z_p r_p, both factors
  rounded: |error| <= 2 2^-8 sum_p |z_p r_p| + 2^-8 |dbeta|, and the sum of absolute terms may
  be far above |dbeta| (with one token and 16 columns, as here, it is).
"""
import numpy as np
import pytest
import torch

import delta_ref as ref
import ssd_chunked_scan_03_amd as ssd

pytestmark = pytest.mark.gpu

F32 = 384 * 2.0 ** -24
B16 = 2.0 ** -8
GRAD_TOL = dict(dx=1, dC=2, dB=3)


def up(d):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def check_y(y, yr, w, dtype, where):
    got = y.double().cpu()
    assert torch.isfinite(got).all(), where
    lim = (B16 if dtype == "bf16" else F32) * (yr.abs() + w) + (F32 * w if dtype == "bf16" else 0)
    worst = ((got - yr).abs() / lim.clamp(min=1e-30)).max().item() if got.numel() else 0.0
    assert worst <= 1.0, (where, worst)


def forward(d, poison=True, **kw):
    g = up(d)
    b, T, H, P = g["x"].shape
    G, N = g["B"].shape[2:]
    prob = ssd.make_problem(b, T, H, P, N, G, 64, ssd._dtype_code(g["x"]))
    y = torch.full_like(g["x"], float("nan"))
    hT = torch.full((b, H, P, N), float("nan"), device="cuda")
    ws = torch.full((max(1, ssd.delta_workspace_bytes(prob)),), 0xFF, dtype=torch.uint8, device="cuda")
    ssd.delta_fwd_into(prob, g["x"], g["dt"], g["A"], g["B"], g["C"], g["beta"], g["h0"], y, hT, ws)
    torch.cuda.synchronize()
    return y, hT


def check_forward(d, dtype, where, terms=1.0):
    print(f"[delta forward] {where}", flush=True)
    y, hT = forward(d)
    yr, hr, w = ref.walk(d, weights=True)
    check_y(y, yr, w, dtype, where)
    e = ref.rel(hT, hr)
    assert e < F32 * terms, (where, e)


# b, T, H, P, N, G, dtype
FORWARD = [
    (1, 1, 1, 16, 16, 1, "bf16"),
    (1, 1, 2, 16, 16, 1, "f32"),
    (2, 63, 4, 64, 64, 2, "bf16"),
    (2, 64, 4, 32, 32, 1, "bf16"),
    (1, 65, 3, 128, 128, 3, "bf16"),
    (2, 200, 6, 64, 128, 2, "bf16"),
    (1, 257, 2, 128, 256, 1, "bf16"),
    (3, 130, 5, 16, 128, 5, "bf16"),
    (1, 100, 2, 32, 16, 2, "bf16"),
    (2, 129, 4, 64, 64, 4, "f32"),
    (1, 70, 2, 128, 256, 2, "f32"),
    (1, 190, 3, 16, 32, 1, "f32"),
    (1, 333, 2, 32, 128, 1, "f32"),
    (2, 150, 140, 64, 64, 2, "bf16"),  # enough chains for the widest slices
    # two column tiles a team
    (1, 130, 80, 64, 128, 8, "bf16"),
    (1, 70, 40, 128, 64, 2, "bf16"),
    # a wave per 16 or 32 columns: headdim 128, few and many chains, narrow heads, dstate 256
    (1, 130, 80, 128, 128, 4, "bf16"),
    (1, 70, 160, 128, 64, 160, "bf16"),
    (1, 130, 160, 64, 128, 8, "bf16"),
    (2, 70, 150, 32, 64, 2, "bf16"),
    (1, 70, 260, 16, 128, 4, "bf16"),
    (2, 70, 264, 64, 128, 8, "bf16"),
    (2, 200, 264, 32, 64, 3, "bf16"),
    (1, 130, 80, 64, 256, 8, "bf16"),
    (1, 70, 40, 128, 256, 5, "bf16"),
    (2, 70, 260, 16, 256, 1, "bf16"),
    # float32 and dstate 16, 32 with full work-groups
    (2, 70, 132, 64, 32, 2, "f32"),
    (1, 130, 260, 64, 128, 4, "f32"),
    (2, 70, 132, 64, 32, 2, "bf16"),
]


@pytest.mark.parametrize("case", FORWARD, ids=lambda c: "b{}T{}H{}P{}N{}G{}{}".format(*c))
def test_forward_matches_definition(case):
    b, T, H, P, N, G, dtype = case
    check_forward(ref.make(b, T, H, P, N, G, 100 + T, dtype), dtype, case)


@pytest.mark.parametrize("kw", [dict(beta="zeros"), dict(beta=1.0), dict(beta=0.0), dict(beta=2.0, dt_hi=1e-3),
                                dict(key="same", beta=1.0, dt_hi=1e-4), dict(key="same", beta=2.0, dt_hi=1e-4),
                                dict(dt_hi=0.0), dict(dt_hi=30.0), dict(h0=False)],
                         ids=lambda k: "-".join(f"{a}{v}" for a, v in k.items()))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_edges(kw, dtype):
    """No write, whole erase, the reflecting limit beta = 2, equal keys without decay (every
    token couples to every other), no decay, decay to nothing within one token, no h0."""
    d = ref.make(2, 150, 2, 32, 64, 1, 7, dtype, **kw)
    terms = 1.0
    if kw.get("key") == "same" and kw["beta"] == 2.0:
        # |B|^2 = 0.98, so S_ij = 0.98 (1 - 2 0.98)^(i-j-1) and the terms of a residual's sum reach
        # sum_j beta |S_ij| = 1.96 (1 - 0.96^63) / 0.04 = 45 times the values themselves
        d["B"] = (d["B"].float() * 0.99).to(d["B"].dtype)
        terms = 46.0
    check_forward(d, dtype, (kw, dtype), terms)


@pytest.mark.parametrize("case", [(2, 130, 4, 64, 128, 2), (1, 130, 160, 64, 128, 8), (1, 130, 2, 64, 256, 1),
                                  (1, 130, 80, 64, 256, 1), (1, 130, 2, 32, 32, 1), (1, 130, 160, 64, 64, 8)],
                         ids=lambda c: "b{}T{}H{}P{}N{}G{}".format(*c))
@pytest.mark.parametrize("key", ["unit", "same"])
def test_y_is_good_to_its_own_rounding(case, key):
    """The bfloat16 y against the exact one: its own rounding's mean square, and beside it only what
    products in two terms leave, 3 2^-17 of each term.  Those roundings are independent and each y
    has N terms a state column and more, so their squares add to (3 2^-17 w)^2 / N at most in the
    mean, w the sum of absolute terms."""
    b, T, H, P, N, G = case
    d = ref.make(b, T, H, P, N, G, 31, "bf16", key=key, dt_hi=0.02)
    y, _ = forward(d)
    yr, _, w = ref.walk(d, weights=True)
    own = (yr.to(torch.bfloat16).double() - yr).square().sum()
    rest = (3 * 2.0 ** -17 * w).square().sum() / N
    assert (y.double().cpu() - yr).square().sum() < 1.02 * (own + rest), (case, key)


def test_strong_gates_keep_the_ratio_of_neighbours():
    """One token with a decay of e^-3000 in the middle of a chunk of weak ones: the decay sums
    behind it are thousands, their differences 1e-3."""
    d = ref.make(1, 128, 2, 16, 32, 1, 8, "f32", dt_hi=1e-3)
    d["dt"][:, 20] = 3000.0 / d["A"].abs()
    check_forward(d, "f32", "gate")


def test_state_carries_over_calls():
    """Two halves, the second from the first's hT, against the whole."""
    d = ref.make(2, 260, 4, 64, 64, 2, 9, "bf16")
    cut = lambda lo, hi: {k: (v[:, lo:hi].contiguous() if k in ("x", "dt", "B", "C", "beta") else v) for k, v in d.items()}  # noqa: E731
    y0, h0 = forward(cut(0, 101))
    y1, h1 = forward(dict(cut(101, 260), h0=h0.cpu()))
    yr, hr, w = ref.walk(d, weights=True)
    check_y(torch.cat([y0, y1], 1), yr, w, "bf16", "halves")
    assert ref.rel(h1, hr) < F32


def test_empty_sequence_and_batch():
    d = ref.make(2, 0, 4, 32, 32, 2, 10, "bf16")
    y, hT = ssd.delta_fwd(*(up(d)[k] for k in ("x", "dt", "A", "B", "C", "beta", "h0")))
    assert y.shape == (2, 0, 4, 32) and torch.equal(hT.cpu(), d["h0"])
    d = ref.make(0, 5, 4, 32, 32, 2, 10, "bf16")
    y, hT = ssd.delta_fwd(*(up(d)[k] for k in ("x", "dt", "A", "B", "C", "beta", "h0")))
    assert y.shape == (0, 5, 4, 32) and hT.shape == (0, 4, 32, 32)


@pytest.mark.parametrize("lengths,shape,dtype", [
    ([5], (4, 64, 64, 2), "bf16"),
    ([0, 1, 63, 0, 64, 65, 130, 0], (4, 64, 128, 1), "bf16"),
    ([3, 200, 1, 1, 1, 77], (2, 32, 32, 2), "f32"),
    ([0, 0, 0], (2, 16, 16, 1), "bf16"),
    ([0, 1, 63, 0, 64, 65, 130, 0], (40, 128, 128, 4), "bf16"),  # a wave per 16 columns
    ([70, 0, 129], (40, 64, 256, 2), "bf16"),
])
def test_packed_sequences(lengths, shape, dtype):
    """Each sequence is its own walk; tokens outside every sequence keep y as it was, and
    NaN there reaches nothing."""
    H, P, N, G = shape
    T, pad = sum(lengths), 7
    d = ref.make(1, T + 2 * pad, H, P, N, G, 11, dtype)
    for k in ("x", "B", "C", "beta", "dt"):
        d[k][:, :pad] = float("nan")
        d[k][:, T + pad:] = float("nan")
    g = torch.Generator().manual_seed(3)
    h0 = 0.1 * torch.randn(len(lengths), H, P, N, generator=g)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]) + pad, dtype=torch.int32)
    v = up({k: d[k][0].contiguous() for k in ("x", "dt", "B", "C", "beta")})
    prob = ssd.make_problem(len(lengths), T + 2 * pad, H, P, N, G, 64, ssd._dtype_code(v["x"]))
    y = torch.full_like(v["x"], 7.0)
    hT = torch.full((len(lengths), H, P, N), float("nan"), device="cuda")
    ws = torch.full((ssd.delta_workspace_bytes(prob, True),), 0xFF, dtype=torch.uint8, device="cuda")
    print(f"[delta packed] {lengths} {shape} {dtype}", flush=True)
    ssd.delta_fwd_varlen_into(prob, cu.cuda(), v["x"], v["dt"], d["A"].cuda(), v["B"], v["C"], v["beta"], h0.cuda(), y,
                              hT, ws)
    torch.cuda.synchronize()
    assert (y[:pad] == 7.0).all() and (y[T + pad:] == 7.0).all()
    for s, n in enumerate(lengths):
        lo = int(cu[s])
        one = {k: d[k][:, lo:lo + n] for k in ("x", "dt", "B", "C", "beta")}
        yr, hr, w = ref.walk(dict(one, A=d["A"], h0=h0[s:s + 1]), weights=True)
        check_y(y[lo:lo + n][None], yr, w, dtype, (lengths, s))
        assert ref.rel(hT[s:s + 1], hr) < F32, (lengths, s)


@pytest.mark.parametrize("rows", [200, 1100])
def test_many_packed_sequences(rows):
    """More rows than one wave's lanes, put in order by length, and more than are put in order: each
    against the dense call on its own tokens."""
    g = torch.Generator().manual_seed(41)
    lens = torch.randint(0, 40, (rows,), generator=g)
    lens[rows // 2], lens[rows - 1] = 700, 130
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)])
    T = int(cu[-1])
    d = up(ref.make(1, T, 2, 32, 64, 1, 42, "bf16"))
    h0 = 0.1 * torch.randn(rows, 2, 32, 64, generator=g).cuda()
    t = {k: d[k][0].contiguous() for k in ("x", "dt", "B", "C", "beta")}
    y, hT = ssd.delta_fwd_varlen(t["x"], t["dt"], d["A"], t["B"], t["C"], t["beta"], cu.int().cuda(), h0)
    for r in [0, 1, 63, 64, rows // 2, rows - 2, rows - 1]:
        lo, hi = int(cu[r]), int(cu[r + 1])
        cut = {k: d[k][:, lo:hi].contiguous() for k in t}
        y1, h1 = ssd.delta_fwd(cut["x"], cut["dt"], d["A"], cut["B"], cut["C"], cut["beta"], h0[r:r + 1])
        # (the few rows of the dense call may run in teams: sums in another order, y a rounding apart)
        assert ref.rel(hT[r:r + 1], h1.cpu().double()) < F32, r
        if hi > lo:
            assert ref.rel(y[None, lo:hi], y1.cpu().double()) < B16, r


def test_packed_offsets_outside_the_axis_stay_in_bounds():
    """Offsets are clamped into the axis and made nondecreasing: any values are memory-safe."""
    d = ref.make(1, 100, 2, 32, 32, 1, 12, "bf16")
    v = up({k: d[k][0].contiguous() for k in ("x", "dt", "B", "C", "beta")})
    cu = torch.tensor([0, 90, 40, 1000], dtype=torch.int32, device="cuda")
    y, hT = ssd.delta_fwd_varlen(v["x"], v["dt"], d["A"].cuda(), v["B"], v["C"], v["beta"], cu)
    torch.cuda.synchronize()
    assert torch.isfinite(y.float()).all() and torch.isfinite(hT).all()


STEP = [(1, 1, 2, 16, 16, 1, "f32"), (3, 1, 8, 64, 128, 2, "bf16"), (2, 5, 6, 32, 256, 3, "f32"),
        (2, 7, 4, 128, 64, 1, "bf16"), (8, 1, 80, 64, 128, 1, "bf16")]


@pytest.mark.parametrize("case", STEP, ids=lambda c: "b{}T{}H{}P{}N{}G{}{}".format(*c))
def test_step_matches_definition(case):
    b, T, H, P, N, G, dtype = case
    d = ref.make(b, T, H, P, N, G, 200 + T, dtype)
    g = up(d)
    h = g["h0"].clone()
    y = ssd.delta_step(g["x"], g["dt"], g["A"], g["B"], g["C"], g["beta"], h)
    yr, hr, w = ref.walk(d, weights=True)
    check_y(y, yr, w, dtype, case)
    assert ref.rel(h, hr) < F32


def test_step_continues_the_chunked_walk():
    d = ref.make(2, 140, 4, 64, 64, 2, 13, "bf16")
    cut = lambda lo, hi: {k: (v[:, lo:hi].contiguous() if k in ("x", "dt", "B", "C", "beta") else v) for k, v in d.items()}  # noqa: E731
    _, h = forward(cut(0, 133))
    g = up(cut(133, 140))
    y = ssd.delta_step(g["x"], g["dt"], g["A"], g["B"], g["C"], g["beta"], h)
    yr, hr, w = ref.walk(d, weights=True)
    check_y(y, yr[:, 133:], w[:, 133:], "bf16", "continue")
    assert ref.rel(h, hr) < F32


def test_step_without_tokens_keeps_the_state():
    d = ref.make(2, 0, 4, 32, 32, 2, 14, "bf16")
    g = up(d)
    h = g["h0"].clone()
    ssd.delta_step(g["x"], g["dt"], g["A"], g["B"], g["C"], g["beta"], h)
    assert torch.equal(h, g["h0"])


def backward(d, gr, poison=True):
    g, e = up(d), up(gr)
    b, T, H, P = g["x"].shape
    G, N = g["B"].shape[2:]
    prob = ssd.make_problem(b, T, H, P, N, G, 64, ssd._dtype_code(g["x"]))
    out = {n: torch.full_like(g[k], float("nan")) for n, k in ref.GRAD_OF.items() if n != "dh0"}
    out["dh0"] = torch.full((b, H, P, N), float("nan"), device="cuda")
    ws = torch.full((max(1, ssd.delta_bwd_workspace_bytes(prob)),), 0xFF, dtype=torch.uint8, device="cuda")
    ssd.delta_bwd_into(prob, g["x"], g["dt"], g["A"], g["B"], g["C"], g["beta"], g["h0"], e["dy"], e["dhT"], out["dx"],
                       out["ddt"], out["dA"], out["dB"], out["dC"], out["dbeta"], out["dh0"], ws)
    torch.cuda.synchronize()
    return out


def check_backward(d, gr, dtype, where):
    print(f"[delta backward] {where}", flush=True)
    out, want = backward(d, gr), ref.grads(d, gr)
    worst = {}
    for n in out:
        tol = F32 + (GRAD_TOL[n] * B16 if dtype == "bf16" and n in GRAD_TOL else 0.0)
        worst[n] = ref.rel(out[n], want[n]) / tol
    if dtype == "bf16":
        terms = (want["dx"] / d["beta"].double()[..., None] * ref.residuals(d)).abs().sum(-1)
        lim = B16 * (2 * terms + want["dbeta"].abs()) + F32 * terms
        worst["dbeta"] = ((out["dbeta"].double().cpu() - want["dbeta"]).abs() / lim).max().item()
    assert all(v <= 1.0 for v in worst.values()), (where, worst)
    return out


BACKWARD = [
    (1, 1, 1, 16, 16, 1, "bf16"),
    (1, 1, 2, 16, 16, 1, "f32"),
    (2, 63, 4, 64, 64, 2, "bf16"),
    (1, 129, 4, 32, 128, 1, "bf16"),
    (2, 130, 3, 128, 128, 3, "bf16"),
    (1, 70, 2, 128, 256, 1, "bf16"),
    (1, 200, 6, 16, 32, 2, "bf16"),
    (2, 133, 4, 64, 64, 2, "f32"),
    (1, 65, 2, 128, 256, 2, "f32"),
    (1, 90, 3, 16, 16, 1, "f32"),
    (1, 1100, 2, 16, 32, 1, "f32"),   # a long sum into dA
    # two column tiles a team; dstate 256 with more teams than CUs; full work-groups
    (1, 130, 80, 64, 128, 8, "bf16"),
    (1, 70, 40, 128, 64, 2, "bf16"),
    (2, 70, 40, 128, 128, 1, "bf16"),
    (1, 70, 80, 64, 256, 8, "bf16"),
    (2, 70, 132, 64, 32, 2, "f32"),
    (2, 70, 132, 64, 32, 2, "bf16"),
]


@pytest.mark.parametrize("case", BACKWARD, ids=lambda c: "b{}T{}H{}P{}N{}G{}{}".format(*c))
def test_backward_matches_reverse_mode(case):
    b, T, H, P, N, G, dtype = case
    check_backward(ref.make(b, T, H, P, N, G, 300 + T, dtype), ref.make_grads(b, T, H, P, N, 300 + T, dtype), dtype, case)


@pytest.mark.parametrize("kw", [dict(beta="zeros"), dict(beta=1.0), dict(beta=0.0), dict(key="same", beta=1.0, dt_hi=1e-4),
                                dict(dt_hi=0.0), dict(h0=False)],
                         ids=lambda k: "-".join(f"{a}{v}" for a, v in k.items()))
def test_backward_edges(kw):
    d = ref.make(2, 100, 2, 32, 64, 1, 17, "f32", **kw)
    check_backward(d, ref.make_grads(2, 100, 2, 32, 64, 17, "f32"), "f32", kw)


def test_backward_without_dhT():
    d, gr = ref.make(1, 80, 2, 32, 32, 1, 18, "f32"), ref.make_grads(1, 80, 2, 32, 32, 18, "f32")
    gr["dhT"] = None
    check_backward(d, gr, "f32", "no dhT")


def test_backward_against_differences():
    """<gradient, direction> of every input against the central difference of the float64 loss
    along it: differences of size e are off by about e^2 times the third derivative."""
    d, gr = ref.make(1, 70, 2, 16, 32, 1, 19, "f32"), ref.make_grads(1, 70, 2, 16, 32, 19, "f32")
    out = backward(d, gr)
    loss = lambda v: ((lambda yh: (yh[0] * gr["dy"].double()).sum() + (yh[1] * gr["dhT"].double()).sum())(ref.walk(v))).item()  # noqa: E731
    g = torch.Generator().manual_seed(20)
    for n, k in ref.GRAD_OF.items():
        v = torch.randn(d[k].shape, generator=g, dtype=torch.float64)
        v = v * d[k].double().abs().clamp(min=1e-3)  # small beside the value itself
        e = 1e-4
        diff = (loss(dict(d, **{k: d[k].double() + e * v})) - loss(dict(d, **{k: d[k].double() - e * v}))) / (2 * e)
        got = (out[n].double().cpu() * v).sum().item()
        scale = (out[n].double().cpu() * v).norm().item()
        assert abs(got - diff) < 1e-4 * max(scale, abs(diff)) + 1e-6, (n, got, diff)


def test_backward_is_deterministic_and_without_tokens():
    d, gr = ref.make(2, 300, 8, 64, 64, 1, 21, "bf16"), ref.make_grads(2, 300, 8, 64, 64, 21, "bf16")
    a, b = backward(d, gr), backward(d, gr)
    assert all(torch.equal(a[k], b[k]) for k in a)
    d, gr = ref.make(2, 0, 4, 32, 32, 2, 22, "bf16"), ref.make_grads(2, 0, 4, 32, 32, 22, "bf16")
    out = backward(d, gr)
    assert torch.equal(out["dh0"].cpu(), gr["dhT"]) and (out["dA"] == 0).all()


def _capture(run):
    run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    return g


def test_graph_replays_match_eager():
    """A training step's calls (norm, forward, backward) and a decode step captured together;
    every replay, with eager work between, gives the eager results bit for bit."""
    b, T, H, P, N, G = 2, 150, 4, 64, 64, 2
    d, gr = up(ref.make(b, T, H, P, N, G, 23, "bf16")), up(ref.make_grads(b, T, H, P, N, 23, "bf16"))
    freq = (10000.0 ** (-torch.arange(16, device="cuda") / 16)).float()
    kw = dict(mode="l2", inv_freq=freq)
    out = {}
    h = torch.zeros_like(d["h0"])

    def run():
        y, hT = ssd.delta_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["beta"], d["h0"], norm=kw)
        g = ssd.delta_bwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["beta"], gr["dy"], d["h0"], gr["dhT"], norm=kw)
        h.copy_(hT)
        ys = ssd.delta_step(d["x"], d["dt"], d["A"], d["B"], d["C"], d["beta"], h, norm=kw)
        out.update(y=y, hT=hT, ys=ys, h=h, **g)

    run()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in out.items()}
    graph = _capture(run)
    for r in range(4):
        for v in out.values():
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for k, v in out.items():
            assert torch.equal(v, want[k]), (r, k)
        a = torch.randn(1 << 20, device="cuda")
        float((a * a).sum())
        torch.cuda.synchronize()


def test_packed_graph_follows_new_offsets():
    """A captured packed call reads its offsets when it is replayed: other lengths in the same tensor
    give what the eager call gives on them."""
    d = up(ref.make(1, 400, 40, 128, 128, 4, 25, "bf16"))
    t = [d[k][0].contiguous() for k in ("x", "dt")] + [d["A"]] + [d[k][0].contiguous() for k in ("B", "C", "beta")]
    offsets = [[0, 10, 300, 300, 400], [0, 200, 210, 390, 400], [0, 0, 0, 0, 400]]
    cu = torch.tensor(offsets[0], dtype=torch.int32, device="cuda")
    out = {}

    def run():
        out["y"], out["hT"] = ssd.delta_fwd_varlen(*t, cu)

    run()
    torch.cuda.synchronize()
    graph = _capture(run)
    for r in range(4):
        cu.copy_(torch.tensor(offsets[r % 3], dtype=torch.int32))
        want = ssd.delta_fwd_varlen(*t, cu)
        for v in out.values():
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["y"], want[0]) and torch.equal(out["hT"], want[1]), r


def test_on_a_side_stream():
    d = up(ref.make(2, 150, 4, 64, 64, 2, 24, "bf16"))
    args = [d[k] for k in ("x", "dt", "A", "B", "C", "beta", "h0")]
    y0, h0 = ssd.delta_fwd(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y1, h1 = ssd.delta_fwd(*args)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(h0, h1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_of_norm_rule_and_decode(dtype):
    """The operators together, as a layer runs them: B and C from one projection normed and
    turned, the chunked rule over the prompt, then decode steps at the following positions,
    against the definitions over all tokens; and the backward through the norm."""
    b, T, T1, H, P, N, G = 2, 96, 90, 4, 32, 64, 2
    d = ref.make(b, T, H, P, N, G, 25, dtype)
    g = torch.Generator().manual_seed(26)
    proj = (torch.randn(b, T, 2 * G * N, generator=g) * 2).to(d["x"].dtype)
    Br, Cr = proj[..., :G * N].unflatten(-1, (G, N)), proj[..., G * N:].unflatten(-1, (G, N))
    freq = (1000.0 ** (-torch.arange(16) / 16)).float()
    wC = torch.randn(N, generator=g)
    pos = torch.arange(T, dtype=torch.int32).expand(b, T).contiguous()
    dev = up(d)
    pj = proj.cuda()
    Bd, Cd = pj[..., :G * N].unflatten(-1, (G, N)), pj[..., G * N:].unflatten(-1, (G, N))
    kw = dict(mode="l2", inv_freq=freq.cuda(), wC=wC.cuda())
    # the values the rule sees are the norm's outputs as rounded
    Bn, Cn = ssd.bc_norm(Bd, Cd, **kw)
    cut = lambda v, lo, hi: v[:, lo:hi].contiguous()  # noqa: E731
    y0, h = ssd.delta_fwd(*(cut(dev[k], 0, T1) for k in ("x", "dt")), dev["A"], Bd[:, :T1].contiguous(),
                          Cd[:, :T1].contiguous(), cut(dev["beta"], 0, T1), dev["h0"],
                          norm=dict(kw, positions=pos[:, :T1].contiguous().cuda()))
    ys = [y0]
    for t in range(T1, T):
        # a decode step's B and C are views into that token's projection
        ys.append(ssd.delta_step(*(cut(dev[k], t, t + 1) for k in ("x", "dt")), dev["A"], Bd[:, t:t + 1], Cd[:, t:t + 1],
                                 cut(dev["beta"], t, t + 1), h, norm=dict(kw, positions=pos[:, t:t + 1].contiguous().cuda())))
    n = dict(d, B=Bn.cpu(), C=Cn.cpu())
    yr, hr, w = ref.walk(n, weights=True)
    check_y(torch.cat(ys, 1), yr, w, dtype, "layer")
    assert ref.rel(h, hr) < F32
    if dtype == "f32":
        gr = ref.make_grads(b, T, H, P, N, 27, dtype)
        e = up(gr)
        out = ssd.delta_bwd(dev["x"], dev["dt"], dev["A"], Bd, Cd, dev["beta"], e["dy"], dev["h0"], e["dhT"], norm=kw)
        f = {k: v.double().clone().requires_grad_() for k, v in dict(B=Br, C=Cr, w=wC).items()}
        nb = ref.norm(f["B"], None, "l2", 1e-6, freq, pos, False)
        nc = ref.norm(f["C"], f["w"], "l2", 1e-6, freq, pos, False)
        y, hT = ref.walk(dict(d, B=nb, C=nc))
        loss = (y * gr["dy"].double()).sum() + (hT * gr["dhT"].double()).sum()
        want = torch.autograd.grad(loss, [f["B"], f["C"], f["w"]])
        for k, v in zip(("dB", "dC", "dwC"), want):
            assert ref.rel(out[k], v) < 2 * F32, k  # two operators' float32 sums
        assert "dwB" not in out
