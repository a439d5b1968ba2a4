"""What the operators on a pool of states refuse, on the host: the C ABI before any HIP call (the fake
device addresses are never dereferenced) and the Python binding before the C ABI; and that the
float64 reference of their GPU tests agrees with other forms of itself."""
import ctypes

import pytest
import torch

import pool_ref as ref
import ssd_chunked_scan_03_amd as ssd

OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE, ALIGN, ALIAS = range(7)
SP = 1 << 30  # distance between fake tensors
b, T, H, P, N, G, S = 3, 9, 4, 32, 64, 2, 7

STEP = "x dt A B C D beta pool slots out y"
TREE = "x dt A B C D beta parents pool slots y"
COMMIT = "x dt A B beta parents last pool slots out"
CALLS = {"ssd_pool_step": (STEP, "x dt A B C pool slots y", "pool y"),
         "ssd_tree_step": (TREE, "x dt A B C parents pool slots y", "y"),
         "ssd_tree_commit": (COMMIT, "x dt A B parents last pool slots", "pool")}


def prob(**kw):
    v = dict(b=b, T=T, H=H, P=P, N=N, G=G, xs=None, bs=None, cs=None, S=S, ss=None, dtype=ssd.SSD_BF16, flags=0)
    v.update(kw)
    rows = v["H"] * v["P"], v["G"] * v["N"]
    return ssd.PoolProblem(v["b"], v["T"], v["H"], v["P"], v["N"], v["G"], rows[0] if v["xs"] is None else v["xs"],
                           rows[1] if v["bs"] is None else v["bs"], rows[1] if v["cs"] is None else v["cs"], v["S"],
                           rows[0] * v["N"] if v["ss"] is None else v["ss"], v["dtype"], v["flags"])


def names(name, rule="scan"):
    """Every operand at an address of its own, without the other rule's."""
    return {n: 0 if n == ("beta" if rule == "scan" else "D") else SP * (i + 1) for i, n in enumerate(CALLS[name][0].split())}


def go(name, p, args):
    a = [ctypes.c_void_p(v) if v else None for v in args.values()]
    return getattr(ssd._load(), name)(ctypes.byref(p) if p is not None else None, *a, None)


@pytest.mark.parametrize("rule", ["scan", "delta"])
@pytest.mark.parametrize("name", list(CALLS))
def test_bad_calls_are_refused(name, rule):
    every, needed, outs = names(name, rule), CALLS[name][1], CALLS[name][2]
    for n in needed.split():
        assert go(name, prob(), dict(every, **{n: 0})) == NULL, n
    assert go(name, None, every) == NULL
    for kw in (dict(H=6, G=4), dict(H=0), dict(G=0), dict(b=-1), dict(T=-1), dict(S=-1), dict(P=0), dict(N=-16),
               dict(xs=H * P - 8), dict(bs=G * N - 8), dict(ss=H * P * N - 4), dict(xs=0)):
        assert go(name, prob(**kw), every) == SHAPE, kw
    for kw in (dict(P=48), dict(N=512), dict(P=256), dict(N=8), dict(dtype=5), dict(dtype=-1), dict(flags=1),
               dict(H=1 << 24, G=1), dict(b=1 << 24), dict(b=1 << 23, H=4), dict(xs=(1 << 32) + 8),
               dict(bs=(1 << 40)), dict(S=1 << 31), dict(S=1 << 20, ss=1 << 30), dict(ss=1 << 41),
               dict(b=1 << 13, T=256 if "tree" in name else 1 << 24, xs=1 << 32)):
        assert go(name, prob(**kw), every) == UNSUPPORTED, kw
    assert go(name, prob(H=1 << 18, P=128, G=1), every) == UNSUPPORTED  # (16 nodes of y within 2 GiB)
    if "tree" in name:
        assert go(name, prob(T=257), every) == UNSUPPORTED
    if name != "ssd_tree_commit":
        assert go(name, prob(cs=G * N - 8), every) == SHAPE
        assert go(name, prob(), dict(every, D=SP * 20, beta=SP * 21)) == UNSUPPORTED
    for n, v in every.items():
        if v:
            assert go(name, prob(), dict(every, **{n: v + 1})) == ALIGN, n
    for n in "x B C y pool".split():
        if n in every:
            assert go(name, prob(), dict(every, **{n: every[n] + 8})) == ALIGN, n
    for kw in (dict(xs=H * P + 4), dict(bs=G * N + 4), dict(ss=H * P * N + 2)):
        assert go(name, prob(**kw), every) == ALIGN, kw
    for n in outs.split():
        for other, v in every.items():
            if other != n and v:
                assert go(name, prob(), dict(every, **{n: v})) == ALIAS, (n, other)
    if name == "ssd_tree_step":  # (the pool is read: it may hold an input)
        assert go(name, prob(), dict(every, y=every["pool"] + 4 * (S - 1) * H * P * N)) == ALIAS


def test_strides_reach_as_far_as_they_say():
    """An output behind the last token of a strided input does not overlap it, one on that token does."""
    every = names("ssd_tree_step")
    p = prob(xs=H * P + 64)
    last = every["x"] + ((b * T - 1) * (H * P + 64) + H * P) * 2
    assert go("ssd_tree_step", p, dict(every, y=last - 16)) == ALIAS
    p = prob(ss=2 * H * P * N)
    end = every["pool"] + ((S - 1) * 2 * H * P * N + H * P * N) * 4
    assert go("ssd_tree_step", p, dict(every, y=end - 16)) == ALIAS


@pytest.mark.parametrize("name", list(CALLS))
def test_nothing_to_do_enqueues_nothing(name):
    nothing = {n: 0 for n in names(name)}
    assert go(name, prob(b=0), nothing) == OK
    assert go(name, prob(T=0, xs=0), nothing) == OK
    if name != "ssd_tree_step":
        assert go(name, prob(T=0), dict(nothing, out=SP)) == NULL  # (the states have to go to the out slots)


def pages(**kw):
    v = dict(rows=4, layers=3, slots=6, elems=1024, ls=6 * 1024, ss=1024)
    v.update(kw)
    return ssd.Pages(*(v[n] for n in ("rows", "layers", "slots", "elems", "ls", "ss")))


FORK, COMPACT = "pool table sources new", "pool table new count"


@pytest.mark.parametrize("name,every", [("ssd_pool_fork", FORK), ("ssd_pool_compact", COMPACT)])
def test_bad_pages_are_refused(name, every):
    at = {n: SP * (i + 1) for i, n in enumerate(every.split())}
    for n in at:
        assert go(name, pages(), dict(at, **{n: 0})) == NULL, n
        assert go(name, pages(), dict(at, **{n: at[n] + (4 if n == "pool" else 2)})) == ALIGN, n
    assert go(name, None, at) == NULL
    for kw in (dict(rows=-1), dict(layers=-1), dict(slots=-1), dict(elems=0), dict(ss=1020), dict(ls=1020),
               dict(ls=2048), dict(ls=1024, ss=2 * 1024)):
        assert go(name, pages(**kw), at) == SHAPE, kw
    for kw in (dict(slots=16385), dict(rows=65537, slots=16384), dict(layers=65537), dict(elems=1 << 41),
               dict(ls=1 << 41), dict(ss=1 << 41)):
        want = SHAPE if name == "ssd_pool_fork" and kw.get("rows", 0) > 65536 else UNSUPPORTED
        assert go(name, pages(**kw), at) in (want, UNSUPPORTED), kw
    for kw in (dict(elems=1022), dict(ss=1026, ls=8000), dict(ls=6 * 1024 + 2)):
        assert go(name, pages(**kw), at) == ALIGN, kw
    outs = [n for n in at if n in ("pool", "new", "count")]
    for n in outs:
        for other in at:
            if other != n:
                assert go(name, pages(), dict(at, **{n: at[other]})) == ALIAS, (n, other)
    if name == "ssd_pool_fork":
        assert go(name, pages(rows=7), at) == SHAPE
        assert go(name, pages(rows=0), at) == OK


# ---- the Python binding ----
def tensors(**kw):
    d = ref.make(2, 5, 2, 16, 16, 1, 1, **kw)
    d["last"] = torch.zeros(2, dtype=torch.int32)
    return d


def calls(d):
    a = (d["x"], d["dt"], d["A"], d["B"])
    return {"step": lambda: ssd.pool_step(*a, d["C"], d["pool"], d["slots"], D=d["D"], beta=d["beta"], out_slots=d["out_slots"]),
            "tree": lambda: ssd.tree_step(*a, d["C"], d["parents"], d["pool"], d["slots"], D=d["D"], beta=d["beta"]),
            "commit": lambda: ssd.tree_commit(*a, d["parents"], d["last"], d["pool"], d["slots"], beta=d["beta"],
                                              out_slots=d["out_slots"])}


def test_binding_refuses_host_tensors():
    for name, f in calls(tensors()).items():
        with pytest.raises(ValueError, match="GPU tensors"):
            f()
        print(name, "refused")
    d = tensors()
    with pytest.raises(ValueError, match="GPU tensor"):
        ssd.pool_fork(d["pool"], d["slots"], d["slots"])
    with pytest.raises(ValueError, match="GPU tensor"):
        ssd.pool_compact(d["pool"], d["slots"])
    p, q = prob(), pages()
    y, t = torch.empty_like(d["x"]), d["slots"]
    for f in (lambda: ssd.pool_step_into(p, d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], None, d["pool"], t, None, y),
              lambda: ssd.tree_step_into(p, d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], None, d["parents"], d["pool"], t, y),
              lambda: ssd.tree_commit_into(p, d["x"], d["dt"], d["A"], d["B"], None, d["parents"], d["last"], d["pool"], t, None),
              lambda: ssd.pool_fork_into(q, d["pool"], t, t, t.clone()),
              lambda: ssd.pool_compact_into(q, d["pool"], t, t.clone(), t[:1].clone())):
        with pytest.raises(ValueError, match="GPU tensors"):
            f()


def test_binding_refuses_shapes_and_types_first():
    def bad(f, kind, match):
        with pytest.raises(kind, match=match):
            f()

    for name in ("step", "tree", "commit"):
        d = tensors()
        bad(calls(dict(d, x=d["x"][0]))[name], ValueError, r"x must be")
        bad(calls(dict(d, pool=d["pool"][0]))[name], ValueError, "pool")
        bad(calls(dict(d, pool=d["pool"][:, :1]))[name], ValueError, "pool must have shape")
        bad(calls(dict(d, pool=d["pool"].double()))[name], TypeError, "pool must be float32")
        bad(calls(dict(d, x=d["x"].half()))[name], TypeError, "bfloat16 or float32")
        bad(calls(dict(d, B=d["B"].float()))[name], TypeError, "one dtype")
        bad(calls(dict(d, B=d["B"][:, :4]))[name], ValueError, "B must have shape")
        bad(calls(dict(d, slots=None))[name], ValueError, "slots is required")
        bad(lambda: ssd.pool_fork(d["pool"].double(), d["slots"], d["slots"]), TypeError, "float32")
        bad(lambda: ssd.pool_fork(d["pool"][0], d["slots"], d["slots"]), ValueError, "pool must be")
        bad(lambda: ssd.pool_fork(d["pool"], d["slots"], None), ValueError, "sources")


# ---- the reference ----
@pytest.mark.parametrize("rule", ["scan", "delta"])
def test_reference_line_is_the_step(rule):
    """A tree without branches is the recurrence, and its last node's commit its last state."""
    d = ref.make(2, 7, 4, 16, 32, 2, 5, "f32", rule, "line")
    y, pool = ref.step(d)
    assert torch.equal(ref.tree(d), y)
    assert torch.equal(ref.commit(d, [6, 6]), pool)
    assert torch.equal(ref.commit(d, [-1, 7]), d["pool"].double())


def test_reference_tree_is_its_paths():
    """Each node's y equals that of its path alone."""
    d = ref.make(1, 12, 2, 16, 16, 1, 8, "f32", "delta", "holes")
    y = ref.tree(d)
    for k, path in enumerate(ref.paths(d["parents"])[0]):
        if path is None:
            assert not y[0, k].any()
            continue
        one = {n: (d[n][:, path].contiguous() if n in ("x", "dt", "B", "C", "beta") else d[n]) for n in d}
        assert torch.equal(ref.step(one)[0][0, -1], y[0, k])


def test_reference_fork_by_hand():
    pool = torch.arange(6.0).reshape(6, 1, 1, 1).expand(6, 2, 2, 2).clone()
    table = torch.tensor([3, 1, 5, -1], dtype=torch.int32)
    # row 0 goes on, row 1 copies row 0, row 2 begins, row 3 takes over row 2's state
    new, after = ref.fork(pool, table, torch.tensor([0, 0, -2, 2], dtype=torch.int32))
    assert new.tolist() == [3, 0, 1, 5]
    assert after[:, 0, 0, 0].tolist() == [3, 0, 2, 3, 4, 5]
    new, n, after = ref.compact(pool, table)
    assert (new.tolist(), n) == ([0, 1, 2, -1], 3)
    assert after[:, 0, 0, 0].tolist() == [3, 1, 5, 3, 4, 5]
