"""What the gated delta rule and the norm of B and C refuse, on the host: the C ABI before any
HIP call (the fake device addresses are never dereferenced) and the Python binding before
the C ABI; and that the float64 reference of their GPU tests agrees with itself."""
import ctypes

import pytest
import torch

import delta_ref as ref
import ssd_chunked_scan_03_amd as ssd

OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE, ALIGN, ALIAS = range(7)
b, T, H, P, N, G = 2, 130, 4, 32, 64, 2
SP = 1 << 26  # distance between fake tensors


def prob(**kw):
    a = dict(b=b, T=T, H=H, P=P, N=N, G=G, Q=64, dtype=ssd.SSD_BF16, flags=0)
    a.update(kw)
    return ssd.make_problem(a["b"], a["T"], a["H"], a["P"], a["N"], a["G"], a["Q"], a["dtype"], a["flags"])


def call(name, p, args, ws=None, ws_bytes=None):
    a = [ctypes.c_void_p(v) if v else None for v in args.values()]
    if ws is not None or ws_bytes is not None:
        a += [ctypes.c_void_p(ws) if ws else None, ws_bytes]
    return getattr(ssd._load(), name)(ctypes.byref(p) if p is not None else None, *a, None)


def names(text):
    return {n: SP * (i + 1) for i, n in enumerate(text.split())}


FWD = "x dt A B C beta h0 y hT"
VAR = "cu x dt A B C beta h0 y hT"
STEP = "x dt A B C beta h y"
BWD = "x dt A B C beta h0 dy dhT dx ddt dA dB dC dbeta dh0"
CALLS = {"ssd_delta_fwd": (FWD, "x dt A B C beta y", "h0 hT", "y hT"),
         "ssd_delta_fwd_varlen": (VAR, "cu x dt A B C beta y", "h0 hT", "y hT"),
         "ssd_delta_step": (STEP, STEP, "", "h y"),
         "ssd_delta_bwd": (BWD, "x dt A B C beta dy dx ddt dA dB dC dbeta", "h0 dhT dh0", "dx ddt dA dB dC dbeta dh0")}
WS = SP * 64


def bytes_of(name, p):
    lib = ssd._load()
    return {"ssd_delta_fwd": lib.ssd_delta_workspace_bytes, "ssd_delta_fwd_varlen": lib.ssd_delta_varlen_workspace_bytes,
            "ssd_delta_bwd": lib.ssd_delta_bwd_workspace_bytes}[name](ctypes.byref(p))


def go(name, p, args, ws=WS, short=0):
    if name == "ssd_delta_step":
        return call(name, p, args)
    return call(name, p, args, ws, (bytes_of(name, p) or (1 << 30)) - short)


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_calls_are_refused(name):
    every, needed, _, outs = CALLS[name]
    p = prob()
    for n in needed.split():
        assert go(name, p, dict(names(every), **{n: 0})) == NULL, n
    assert go(name, prob(H=6, G=4), names(every)) == SHAPE
    for kw in (dict(P=48), dict(N=512), dict(P=256), dict(dtype=5), dict(flags=1), dict(flags=ssd.SCHEDULE_SPLIT)):
        assert go(name, prob(**kw), names(every)) == UNSUPPORTED, kw
    if name != "ssd_delta_step":
        for q in (128, 256):
            assert go(name, prob(Q=q), names(every)) == UNSUPPORTED
            assert bytes_of(name, prob(Q=q)) == 0
        assert go(name, p, names(every), ws=0) == WORKSPACE
        assert go(name, p, names(every), short=1) == WORKSPACE
        assert go(name, p, names(every), ws=WS + 128) == ALIGN
        for n in outs.split():
            assert go(name, p, dict(names(every), **{n: WS + 256})) == ALIAS, n
    for n in names(every):
        assert go(name, p, dict(names(every), **{n: names(every)[n] + 1})) == ALIGN, n
    for n in outs.split():
        for other in names(every):
            if other != n:
                assert go(name, p, dict(names(every), **{n: names(every)[other]})) == ALIAS, (n, other)


def test_null_problem():
    for name in CALLS:
        args = names(CALLS[name][0])
        assert (call(name, None, args) if name == "ssd_delta_step" else call(name, None, args, WS, 1 << 30)) == NULL


def test_grid_limits():
    for kw in (dict(b=1, T=64 * (1 << 24), H=2, G=1), dict(b=70000)):
        assert go("ssd_delta_fwd", prob(**kw), names(FWD)) == UNSUPPORTED
        assert go("ssd_delta_bwd", prob(**kw), names(BWD)) == UNSUPPORTED
    assert go("ssd_delta_step", prob(b=1 << 40), names(STEP)) == UNSUPPORTED
    assert go("ssd_delta_step", prob(T=1 << 40), names(STEP)) == UNSUPPORTED


def test_workspace_grows_with_the_problem():
    lib = ssd._load()
    for f in (lib.ssd_delta_workspace_bytes, lib.ssd_delta_varlen_workspace_bytes, lib.ssd_delta_bwd_workspace_bytes):
        assert f(ctypes.byref(prob(T=0))) == 0 and f(ctypes.byref(prob(b=0))) == 0 and f(ctypes.byref(prob(P=48))) == 0
        assert 0 < f(ctypes.byref(prob(T=64))) < f(ctypes.byref(prob(T=6400)))


def test_empty_problems():
    assert go("ssd_delta_fwd", prob(b=0), names(FWD)) == OK
    assert call("ssd_delta_step", prob(T=0), names(STEP)) == OK
    a = names(FWD)
    assert go("ssd_delta_fwd", prob(T=0), dict(a, hT=0)) == OK
    assert go("ssd_delta_fwd", prob(T=0), dict(a, hT=a["h0"])) == ALIAS
    e = names(BWD)
    assert go("ssd_delta_bwd", prob(T=0), dict(e, dh0=e["dhT"])) == ALIAS
    assert go("ssd_delta_bwd", prob(T=0), dict(e, dA=0)) == NULL


# ---- the norm ----
NRM = "B C wB wC inv_freq positions Bn Cn"
NBW = "B C wB wC inv_freq positions dBn dCn dB dC dwB dwC"


def nprob(**kw):
    a = dict(batch=2, seqlen=5, bheads=2, cheads=3, dstate=64, pairs=16, bstride=None, cstride=None, eps=1e-6, mode=0,
             interleaved=0, dtype=ssd.SSD_BF16)
    a.update(kw)
    a["bstride"] = a["bheads"] * a["dstate"] if a["bstride"] is None else a["bstride"]
    a["cstride"] = a["cheads"] * a["dstate"] if a["cstride"] is None else a["cstride"]
    return ssd.Norm(**a)


def ncall(p, args, ws=WS, nbytes=1 << 20):
    return call("ssd_bc_norm_bwd", p, args, ws, nbytes) if "dBn" in args else call("ssd_bc_norm", p, args)


@pytest.mark.parametrize("every,needed,outs", [(NRM, "B C inv_freq Bn Cn", "Bn Cn"),
                                               (NBW, "B C inv_freq dBn dCn dB dC", "dB dC dwB dwC")], ids=["fwd", "bwd"])
def test_norm_refusals(every, needed, outs):
    a = names(every)
    for n in needed.split():
        assert ncall(nprob(), dict(a, **{n: 0})) == NULL, n
    for kw, st in ((dict(batch=-1), SHAPE), (dict(bheads=0, cheads=0), SHAPE), (dict(pairs=36), SHAPE),
                   (dict(pairs=-4), SHAPE), (dict(bstride=64), SHAPE), (dict(cstride=0), SHAPE),
                   (dict(dstate=48), UNSUPPORTED), (dict(pairs=6), UNSUPPORTED), (dict(mode=2), UNSUPPORTED),
                   (dict(interleaved=2), UNSUPPORTED), (dict(eps=0.0), UNSUPPORTED), (dict(eps=-1.0), UNSUPPORTED),
                   (dict(eps=float("nan")), UNSUPPORTED), (dict(eps=float("inf")), UNSUPPORTED),
                   (dict(dtype=3), UNSUPPORTED), (dict(seqlen=1 << 24), UNSUPPORTED),
                   (dict(batch=1 << 40), UNSUPPORTED), (dict(bheads=1 << 20), UNSUPPORTED),
                   (dict(bstride=132), ALIGN)):
        assert ncall(nprob(**kw), a) == st, kw
    for n in a:
        assert ncall(nprob(), dict(a, **{n: a[n] + 1})) == ALIGN, n
    for n in outs.split():
        for other in a:
            if other != n:
                assert ncall(nprob(), dict(a, **{n: a[other]})) == ALIAS, (n, other)
    # the span of a strided input reaches past its first row
    assert ncall(nprob(bstride=1024), dict(a, **{outs.split()[0]: a["B"] + 1024 * 2 * 9})) == ALIAS
    assert ncall(None, a) == NULL
    if "dBn" in a:
        assert ncall(nprob(), a, ws=0, nbytes=0) == WORKSPACE
        need = ssd.bc_norm_bwd_workspace_bytes(nprob())
        assert need > 0 and ncall(nprob(), a, nbytes=need - 1) == WORKSPACE
        assert ncall(nprob(), a, ws=WS + 16) == ALIGN


def good(dtype=torch.bfloat16):
    z = lambda *s: torch.zeros(*s, dtype=dtype)  # noqa: E731
    return dict(x=z(b, T, H, P), dt=torch.zeros(b, T, H), A=torch.zeros(H), B=z(b, T, G, N), C=z(b, T, G, N),
                beta=z(b, T, H), h0=torch.zeros(b, H, P, N), dy=z(b, T, H, P), dhT=torch.zeros(b, H, P, N))


BIND = {"fwd": lambda a: ssd.delta_fwd(a["x"], a["dt"], a["A"], a["B"], a["C"], a["beta"], a["h0"]),
        "step": lambda a: ssd.delta_step(a["x"], a["dt"], a["A"], a["B"], a["C"], a["beta"], a["h0"]),
        "bwd": lambda a: ssd.delta_bwd(a["x"], a["dt"], a["A"], a["B"], a["C"], a["beta"], a["dy"], a["h0"], a["dhT"])}


@pytest.mark.parametrize("which", list(BIND))
def test_binding_refuses_malformed_tensors(which):
    a = good()
    bad = [("dt", a["dt"][:, :-1]), ("A", torch.zeros(H, N)), ("B", a["B"].float()), ("C", a["C"][..., :32]),
           ("beta", a["beta"].float()), ("beta", a["beta"][..., :1]), ("h0", a["h0"].to(torch.bfloat16)),
           ("h0", a["h0"][:1])]
    if which == "bwd":
        bad += [("dy", a["dy"].float()), ("dhT", a["dhT"][:, :1])]
    for n, v in bad:
        with pytest.raises((ValueError, TypeError)) as e:
            BIND[which](dict(a, **{n: v}))
        assert "GPU tensor" not in str(e.value), n
    with pytest.raises(TypeError):
        BIND[which](good(torch.float16))
    with pytest.raises(ValueError, match="GPU tensor"):
        BIND[which](a)
    with pytest.raises(ValueError):
        BIND[which](dict(a, x=a["x"][0]))


def test_binding_refuses_malformed_packs_and_norms():
    a = good()
    v = {k: a[k][0] for k in ("x", "dt", "B", "C", "beta")}
    cu = torch.tensor([0, 4, T], dtype=torch.int32)
    f = lambda **kw: ssd.delta_fwd_varlen(**{**dict(v, A=a["A"], cu_seqlens=cu), **kw})  # noqa: E731
    with pytest.raises(TypeError):
        f(cu_seqlens=cu.long())
    with pytest.raises(ValueError, match="h0"):
        f(h0=torch.zeros(3, H, P, N))
    with pytest.raises(ValueError, match="positions"):
        f(norm=dict(inv_freq=torch.zeros(4)))
    with pytest.raises(ValueError, match="GPU tensor"):
        f()
    Bt, w = a["B"], torch.ones(N)
    for kw in (dict(wB=w[:3]), dict(wC=w.to(torch.bfloat16)), dict(mode="layer"), dict(inv_freq=w.double()),
               dict(inv_freq=w[:4], positions=torch.zeros(b, T)), dict(inv_freq=w[:4], positions=torch.zeros(T, dtype=torch.int32))):
        with pytest.raises((ValueError, TypeError)) as e:
            ssd.bc_norm(Bt, Bt, **kw)
        assert "GPU tensor" not in str(e.value)
    with pytest.raises(TypeError):
        ssd.bc_norm(Bt, Bt.float())
    with pytest.raises(ValueError):
        ssd.bc_norm(Bt, Bt[:, :-1])
    with pytest.raises(ValueError, match="GPU tensor"):
        ssd.bc_norm(Bt, Bt)


def test_reference_gradients_against_differences():
    d, gr = ref.make(1, 9, 2, 3, 4, 1, 1, "f32"), ref.make_grads(1, 9, 2, 3, 4, 1, "f32")
    d = {k: v.double() for k, v in d.items()}
    want = ref.grads(d, gr)

    def loss(v):
        y, h = ref.walk(v)
        return ((y * gr["dy"].double()).sum() + (h * gr["dhT"].double()).sum()).item()

    g = torch.Generator().manual_seed(2)
    for n, k in ref.GRAD_OF.items():
        v = torch.randn(d[k].shape, generator=g, dtype=torch.float64)
        diff = (loss(dict(d, **{k: d[k] + 1e-5 * v})) - loss(dict(d, **{k: d[k] - 1e-5 * v}))) / 2e-5
        assert abs((want[n] * v).sum().item() - diff) < 1e-6 * max(1.0, abs(diff)), n


def test_sizes_past_the_kernels_reach_are_refused():
    """A chunk's rows of x, or (backward) the states of its heads, past 2 GiB; more threads than a
    launch takes.  Slightly smaller problems are taken."""
    lib = ssd._load()
    fwd, bwd = lib.ssd_delta_workspace_bytes, lib.ssd_delta_bwd_workspace_bytes
    size = lambda f, **kw: f(ctypes.byref(prob(b=1, T=64, **kw)))  # noqa: E731
    over = 1 << 19
    assert size(fwd, H=over, G=1) == 0 and size(fwd, H=over - 512, G=1) > 0
    states = dict(P=32, N=128, G=1)
    assert size(bwd, H=1 << 18, **states) == 0 and size(bwd, H=(1 << 18) - 64, **states) > 0
    assert size(fwd, H=1 << 18, **states) > 0
    assert fwd(ctypes.byref(prob(b=65535, T=1, H=64, P=128, G=1))) == 0
    assert fwd(ctypes.byref(prob(b=16383, T=1, H=64, P=128, G=1))) > 0
