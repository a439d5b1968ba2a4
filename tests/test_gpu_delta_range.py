"""The gated delta rule outside the decays that training starts from: states that grow, and
gradients of decays so strong that little of a state outlives a token.  Shapes select every
walk; tolerances as in test_gpu_delta unless a test states its own."""
import pytest
import torch

import delta_ref as ref
from delta_decay_ref import decay_gradients
import ssd_chunked_scan_03_amd as ssd
import test_gpu_delta as base
from test_gpu_delta import F32, backward, check_backward, check_forward, forward

pytestmark = pytest.mark.gpu

# b, T, H, P, N, G, dtype: teams of one and two column tiles, dstate 256, the walks of narrow
# states and of float32
SHAPES = [(2, 130, 4, 64, 64, 2, "bf16"), (1, 130, 80, 64, 128, 8, "bf16"), (1, 100, 2, 128, 256, 1, "bf16"),
          (1, 130, 4, 32, 32, 2, "bf16"), (2, 100, 2, 16, 16, 1, "bf16"), (2, 130, 4, 64, 64, 2, "f32"),
          (1, 100, 2, 32, 256, 1, "f32"), (1, 77, 3, 16, 16, 1, "f32")]
NAME = "b{}T{}H{}P{}N{}G{}{}"


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: NAME.format(*c))
def test_growing_states(case):
    """A > 0: a_t = exp(dt A) up to 1.03, the state grows by e^2 over the tokens."""
    b, T, H, P, N, G, dtype = case
    d = ref.make(b, T, H, P, N, G, 51, dtype, dt_hi=0.002)
    d["A"] = d["A"].abs()
    check_forward(d, dtype, case)
    check_backward(d, ref.make_grads(b, T, H, P, N, 51, dtype), dtype, case)


def test_empty_sequences_of_many_states():
    """No tokens and states of more elements than one launch has threads (2^32): hT = h0, or 0; dh0 =
    dhT, dA = 0; of the rule and of the scan."""
    b, H, P, N = 10, 16384, 128, 256
    f32 = dict(dtype=torch.float32, device="cuda")
    x, dt = torch.zeros(b, 0, H, P, dtype=torch.bfloat16, device="cuda"), torch.zeros(b, 0, H, **f32)
    B, beta = torch.zeros(b, 0, 1, N, dtype=torch.bfloat16, device="cuda"), torch.zeros(b, 0, H, dtype=torch.bfloat16, device="cuda")
    A, dA = torch.zeros(H, **f32), torch.empty(H, **f32)
    prob = ssd.make_problem(b, 0, H, P, N, 1, 64, ssd.SSD_BF16)
    src, dst = torch.full((b, H, P, N), 3.0, **f32), torch.empty(b, H, P, N, **f32)
    cu = torch.zeros(b + 1, dtype=torch.int32, device="cuda")
    calls = [
        ("forward", 3.0, lambda: ssd.delta_fwd_into(prob, x, dt, A, B, B, beta, src, x, dst, None)),
        ("forward, no h0", 0.0, lambda: ssd.delta_fwd_into(prob, x, dt, A, B, B, beta, None, x, dst, None)),
        ("packed", 3.0, lambda: ssd.delta_fwd_varlen_into(prob, cu, x[0], dt[0], A, B[0], B[0], beta[0], src, x[0], dst, None)),
        ("backward", 3.0, lambda: ssd.delta_bwd_into(prob, x, dt, A, B, B, beta, None, x, src, x, dt, dA, B, B, beta, dst, None)),
        ("scan", 3.0, lambda: ssd.scan_fwd_into(prob, False, x, dt, A, B, B, None, src, x, dst, None)),
        ("scan backward", 3.0, lambda: ssd.scan_bwd_into(prob, x, dt, A, B, B, None, None, x, src, x, dt, dA, B, B, None, dst, None)),
    ]
    for name, want, call in calls:
        print(f"[empty] {name}", flush=True)
        dst.fill_(float("nan"))
        dA.fill_(float("nan"))
        call()
        assert all(bool((dst[i] == want).all()) for i in range(b)), name
        assert "backward" not in name or bool((dA == 0).all()), name


@pytest.mark.parametrize("case", [(1, 200, 4, 32, 64, 2, "bf16"), (1, 200, 160, 64, 128, 8, "bf16"),
                                  (1, 200, 4, 32, 32, 2, "f32")], ids=lambda c: NAME.format(*c))
@pytest.mark.parametrize("which", ["x", "dt", "beta", "B", "C"])
def test_a_nan_stays_where_the_formulas_take_it(case, which):
    """From its token on it is in everything that depends on it; in its chunk it may also be in
    earlier tokens of the same outputs; other chunks before, heads, groups and (x) headdim columns
    are what they are without it, bit for bit."""
    b, T, H, P, N, G, dtype = case
    d = ref.make(b, T, H, P, N, G, 54, dtype)
    t, h, p = 104, 1, 5  # the second chunk's token 40
    y0, h0 = (v.cpu() for v in forward(d))
    heads = slice(h, h + 1) if which in ("x", "dt", "beta") else slice(0, H // G)  # head 1 is of group 0
    cols = slice(p, p + 1) if which == "x" else slice(0, P)
    at = dict(x=(0, t, h, p), dt=(0, t, h), beta=(0, t, h), B=(0, t, 0, 3), C=(0, t, 0, 3))[which]
    d[which] = d[which].clone()
    d[which][at] = float("nan")
    y, hT = (v.cpu() for v in forward(d))
    reached = torch.zeros(y.shape, dtype=torch.bool)
    reached[:, 64:, heads, cols] = True
    assert torch.equal(y[~reached], y0[~reached])
    state = torch.zeros(hT.shape, dtype=torch.bool)
    if which == "C":  # only that token's answer
        assert torch.isnan(y[:, t, heads]).all()
        reached[:] = False
        reached[:, 64:128, heads] = True
        assert torch.equal(y[~reached], y0[~reached])
    else:
        assert torch.isnan(y[:, t:, heads, cols]).all()
        state[:, heads, cols] = True
        assert torch.isnan(hT[state]).all()
    assert torch.equal(hT[~state], h0[~state])


def strong(case, seed, lo, hi, A):
    b, T, H, P, N, G, dtype = case
    d, gr = ref.make(b, T, H, P, N, G, seed, dtype), ref.make_grads(b, T, H, P, N, seed, dtype)
    g = torch.Generator().manual_seed(seed)
    d["dt"] = lo + (hi - lo) * torch.rand(b, T, H, generator=g)
    if A is not None:
        d["A"] = torch.full((H,), A)
    return d, gr


def check_decay_gradients(d, gr, where):
    """Every token's ddt to F32 of its own absolute terms, every head's dA to F32 of theirs: each
    term is a product of float32 values (in bfloat16 problems sums of three terms) with its decay,
    whose exponent of up to 2^7 is good to 2^-18.  What is left of a state under float32's smallest
    number is nothing."""
    print(f"[delta decay gradients] {where}", flush=True)
    out = backward(d, gr)
    ddt, dA, s = decay_gradients(d, gr)
    lim = F32 * s * d["A"].abs().double() + 1e-30
    worst = ((out["ddt"].double().cpu() - ddt).abs() / lim).max().item()
    limA = F32 * (s * d["dt"].double()).sum((0, 1)) + 1e-30
    worstA = ((out["dA"].double().cpu() - dA).abs() / limA).max().item()
    assert worst <= 1.0 and worstA <= 1.0, (where, worst, worstA)


@pytest.mark.parametrize("span", [(0.0, 0.1, None), (0.5, 1.0, -8.0), (1.0, 4.0, -8.0), (0.0, 30.0, None)],
                         ids=lambda s: "dt{}to{}A{}".format(*s))
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: NAME.format(*c))
def test_gradients_of_strong_decays(case, span):
    """Little of a state outlives a token (e^-8 to e^-32 of it, or nothing), and the gradient of its
    decay is as small: it has to come from terms that carry that factor."""
    check_decay_gradients(*strong(case, 52, *span), (case, span))


@pytest.mark.parametrize("at", [0, 20, 63, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_around_a_gate(at, dtype):
    """One token that forgets everything among weak ones: no term reaches across it, and its own
    dt of 3000 / |A| multiplies into dA whatever it is given."""
    case = (1, 128, 2, 32, 64, 1, dtype)
    d, gr = strong(case, 53, 0.0, 1e-3, None)
    d["dt"][:, at] = 3000.0 / d["A"].abs()
    check_decay_gradients(d, gr, (case, at))


@pytest.mark.parametrize("case", [(16, 380, 65, 16, 16, 1, "bf16"), (8, 390, 65, 16, 32, 1, "f32"), (96, 20, 32, 128, 16, 1, "bf16"),
                                  (24, 130, 48, 64, 16, 2, "bf16")], ids=lambda c: NAME.format(*c))
def test_gradients_of_strong_decays_of_many_heads(case):
    """Enough heads and chunks that a work-group takes several heads (the last one of a group alone)."""
    check_decay_gradients(*strong(case, 55, 0.0, 1.0, None), case)


@pytest.mark.parametrize("case", [(1, 130, 160, 64, 256, 8, "bf16"), (1, 70, 80, 128, 256, 5, "bf16")], ids=lambda c: NAME.format(*c))
def test_dstate_256_with_many_chains(case):
    """A wave per 16 columns at the widest state."""
    b, T, H, P, N, G, dtype = case
    check_forward(ref.make(b, T, H, P, N, G, 57, dtype), dtype, case)


def test_packed_dstate_256_with_many_chains():
    base.test_packed_sequences([70, 0, 129], (64, 64, 256, 2), "bf16")


@pytest.mark.parametrize("case", [(64, 9, 129, 16, 64, 1, "bf16"), (128, 9, 131, 16, 16, 1, "bf16"), (64, 9, 129, 16, 16, 1, "f32"),
                                  (128, 5, 131, 16, 64, 1, "bf16")], ids=lambda c: NAME.format(*c))
def test_tables_of_several_heads_a_wave(case):
    """Enough heads and chunks that a wave of the preparation takes two or four heads, the last one of
    a group fewer."""
    b, T, H, P, N, G, dtype = case
    d = ref.make(b, T, H, P, N, G, 58, dtype)
    check_forward(d, dtype, case)
    check_backward(d, ref.make_grads(b, T, H, P, N, 58, dtype), dtype, case)
