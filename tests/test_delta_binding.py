"""What the delta rule's and the norm's Python binding refuses beside malformed shapes, on the
host: tensors that a kernel could not read."""
import pytest
import torch

import ssd_chunked_scan_03_amd as ssd

b, T, H, P, N, G = 1, 5, 2, 16, 16, 1


def tensors(dtype=torch.bfloat16):
    z = lambda *s: torch.zeros(*s, dtype=dtype)  # noqa: E731
    return dict(x=z(b, T, H, P), dt=torch.zeros(b, T, H), A=torch.zeros(H), B=z(b, T, G, N), C=z(b, T, G, N),
                beta=z(b, T, H), h0=torch.zeros(b, H, P, N))


def test_enqueueing_calls_refuse_host_tensors():
    """The calls that enqueue into the caller's own buffers hand addresses on as they are."""
    t = tensors()
    prob = ssd.make_problem(b, T, H, P, N, G, 64, ssd.SSD_BF16)
    ops = [t[k] for k in ("x", "dt", "A", "B", "C", "beta")]
    y, h, ws = torch.empty_like(t["x"]), torch.empty_like(t["h0"]), torch.empty(1 << 20, dtype=torch.uint8)
    cu = torch.tensor([0, T], dtype=torch.int32)
    e = torch.empty_like
    norm = ssd.Norm(b, T, G, G, N, 0, G * N, G * N, 1e-6, 0, 0, ssd.SSD_BF16)
    v = {k: t[k][0] for k in ("x", "dt", "B", "C", "beta")}
    calls = {
        "fwd": lambda: ssd.delta_fwd_into(prob, *ops, t["h0"], y, h, ws),
        "varlen": lambda: ssd.delta_fwd_varlen_into(prob, cu, v["x"], v["dt"], t["A"], v["B"], v["C"], v["beta"], t["h0"],
                                                    y[0], h, ws),
        "step": lambda: ssd.delta_step_into(prob, *ops, h, y),
        "bwd": lambda: ssd.delta_bwd_into(prob, *ops, t["h0"], y, None, *(e(v) for v in ops[:1] + ops[1:]), e(h), ws),
        "norm": lambda: ssd.bc_norm_into(norm, t["B"], t["C"], None, None, None, None, e(t["B"]), e(t["C"])),
        "norm_bwd": lambda: ssd.bc_norm_bwd_into(norm, t["B"], t["C"], None, None, None, None, e(t["B"]), e(t["C"]),
                                                 e(t["B"]), e(t["C"]), None, None, None),
        "nothing": lambda: ssd.bc_norm_into(norm, *[None] * 8),
    }
    for name, f in calls.items():
        with pytest.raises(ValueError, match="GPU tensors"):
            f()
        print(name, "refused")


def test_a_turned_decode_step_needs_its_position():
    """Without positions a one-token call would be turned as the sequence's first token, wherever
    it stands."""
    t = tensors()
    one = lambda v: v[:, :1].contiguous()  # noqa: E731
    freq = torch.ones(4)
    step = lambda norm: ssd.delta_step(one(t["x"]), one(t["dt"]), t["A"], one(t["B"]), one(t["C"]), one(t["beta"]),  # noqa: E731
                                       t["h0"], norm=norm)
    with pytest.raises(ValueError, match="positions"):
        step(dict(inv_freq=freq))
    for norm in (None, dict(mode="l2"), dict(inv_freq=freq, positions=torch.tensor([[7]], dtype=torch.int32))):
        with pytest.raises(ValueError, match="GPU tensor"):  # (goes on to the next check)
            step(norm)
