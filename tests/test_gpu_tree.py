"""GPU parity of the tree of drafted tokens and its commit with the float64 recurrence node by node;
tolerances are derived in pool_ref (tree_limit) and below."""
import pytest
import torch

import pool_ref as ref
import ssd_chunked_scan_03_amd as ssd

pytestmark = pytest.mark.gpu

# A state after at most T tokens, relative to the largest value on the way: every token rounds the decay
# (its exponent is rounded once, |log2| 2^-24, and 2 for the exponential: at most 26 binary orders with
# the inputs here), the product, the sum over dstate (8 in a lane, 5 across) and the update.
STATE = (26 + 13 + 6) * 2.0 ** -24


def up(d):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def tree(d, **kw):
    g = up(d)
    before = g["pool"].clone()
    y = ssd.tree_step(g["x"], g["dt"], g["A"], g["B"], g["C"], g["parents"], g["pool"], g["slots"], D=g["D"],
                      beta=g["beta"], **kw)
    torch.cuda.synchronize()
    assert torch.equal(before.view(torch.int32), g["pool"].view(torch.int32))
    return y


def check_tree(d, where, y=None):
    print(f"[tree] {where}", flush=True)
    y = tree(d) if y is None else y
    want = ref.tree(d)
    lim = ref.tree_limit(d, want)
    got = y.double().cpu()
    assert torch.isfinite(got).all(), where
    off = (got - want).abs()
    assert ((off <= lim) | (off == 0)).all(), (where, (off / lim.clamp(min=1e-300)).max().item())
    return y


# b, K, H, P, N, G, dtype, kind
TREES = [
    (1, 1, 1, 16, 16, 1, "bf16", "tree"),
    (1, 1, 2, 16, 16, 1, "f32", "tree"),
    (2, 7, 4, 64, 64, 2, "bf16", "tree"),
    (3, 16, 6, 32, 32, 3, "bf16", "line"),
    (2, 17, 4, 128, 128, 1, "bf16", "ragged"),
    (2, 33, 2, 64, 128, 2, "f32", "holes"),
    (1, 64, 5, 64, 128, 5, "bf16", "tree"),
    (2, 65, 2, 16, 256, 1, "bf16", "deep"),
    (1, 100, 2, 128, 64, 2, "bf16", "holes"),
    (1, 129, 1, 32, 128, 1, "f32", "deep"),
    (1, 130, 2, 64, 256, 1, "bf16", "line"),
    (1, 256, 1, 64, 64, 1, "bf16", "line"),
    (1, 256, 1, 128, 256, 1, "bf16", "tree"),
    (1, 256, 1, 128, 32, 1, "f32", "deep"),
    (1, 256, 2, 16, 16, 2, "bf16", "star"),
    (4, 21, 3, 32, 16, 1, "f32", "star"),
    (9, 5, 8, 64, 128, 4, "bf16", "ragged"),
    (1, 3, 48, 64, 128, 1, "bf16", "tree"),
    (2, 40, 2, 128, 256, 2, "f32", "tree"),
]


@pytest.mark.parametrize("rule", ["scan", "delta"])
@pytest.mark.parametrize("case", TREES, ids=lambda c: "b{}K{}H{}P{}N{}G{}{}{}".format(*c))
def test_tree_matches_definition(case, rule):
    b, K, H, P, N, G, dtype, kind = case
    check_tree(ref.make(b, K, H, P, N, G, 300 + K, dtype, rule, kind), (case, rule))


@pytest.mark.parametrize("kw", [dict(dt_hi=0.0), dict(dt_hi=30.0), dict(dt_hi=1e7), dict(key="same", dt_hi=1e-4), dict(D=False)],
                         ids=lambda k: "-".join(f"{a}{v}" for a, v in k.items()))
@pytest.mark.parametrize("rule", ["scan", "delta"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_edges(kw, rule, dtype):
    """No decay, decay to nothing within one node (exponents far past what 24 bits keep of a running
    sum), equal keys without decay, no skip term."""
    check_tree(ref.make(2, 50, 2, 32, 64, 1, 9, dtype, rule, "deep", **kw), (kw, rule, dtype))


@pytest.mark.parametrize("rule", ["scan", "delta"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_absent_nodes_and_idle_rows(rule, dtype):
    """Whatever an absent node holds reaches nothing; it and the nodes below it are zero; a row whose
    slot is no slot is zero."""
    d = ref.make(5, 70, 2, 64, 64, 1, 11, dtype, rule, "holes")
    d["parents"][0, 40:] = -2
    d["parents"][1, 0] = 5            # a first node that names a later one: nothing hangs on it
    d["parents"][1, 69] = 2 ** 31 - 1
    d["parents"][1, 3] = -2 ** 31
    d["slots"][2], d["slots"][3] = -1, d["pool"].shape[0]
    there = torch.tensor([[p is not None for p in row] for row in ref.paths(d["parents"])])
    clean = check_tree(d, (rule, dtype))
    assert not clean[2:4].any() and not clean.cpu()[~there].any()
    for bad in (float("nan"), float("inf"), torch.finfo(torch.float32).min):
        e = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
        for name in ("x", "B", "C", "dt", "beta"):
            if e[name] is not None:
                e[name][~there] = bad
                e[name][2:4] = bad
        e["pool"][[s for s in range(e["pool"].shape[0]) if s not in d["slots"].tolist()]] = bad
        assert torch.equal(tree(e).view(torch.int16 if dtype == "bf16" else torch.int32),
                           clean.view(torch.int16 if dtype == "bf16" else torch.int32)), bad


def below(d, i, k):
    """The nodes of row i whose path holds node k."""
    return [n for n, path in enumerate(ref.paths(d["parents"])[i]) if path is not None and k in path]


@pytest.mark.parametrize("rule", ["scan", "delta"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["x", "B", "C", "dt", "beta"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_a_bad_value_stays_in_its_branch(rule, dtype, name, bad):
    """A NaN or infinity in one node is in that node's y and those below it, and nowhere else (one in C
    only in its own; x reaches its head's column only)."""
    if name == "beta" and rule == "scan":
        pytest.skip("the scan has no beta")
    d = ref.make(2, 80, 4, 64, 64, 2, 13, dtype, rule, "tree")
    clean = tree(d)
    for k in (3, 70):
        e = {n: (v.clone() if isinstance(v, torch.Tensor) else v) for n, v in d.items()}
        hit = torch.zeros(e["x"].shape, dtype=torch.bool)
        where = below(d, 1, k) if name != "C" else [k]
        if name == "x":
            e["x"][1, k, 2, 5] = float(bad)
            hit[1, where, 2, 5] = True
        elif name in ("B", "C"):
            e[name][1, k, 1, 7] = float(bad)
            hit[1, where, 2:] = True
        else:
            e[name][1, k, 2] = float(bad)
            hit[1, where, 2] = True
        y = tree(e).cpu()
        assert torch.equal(y[~hit], clean.cpu()[~hit]), (k, "elsewhere")
        if name == "dt" and bad == "inf":
            assert torch.isfinite(y[hit]).all() or rule == "delta"  # (a decay of exp(-inf) = 0)
        else:
            assert not torch.isfinite(y[hit]).any(), (k, "there")


def wide(t, pad, front=0):
    """t's values as a view into a wider projection."""
    b, T, h, n = t.shape
    big = torch.full((b, T, front + h * n + pad), float("nan"), dtype=t.dtype)
    big[..., front:front + h * n] = t.flatten(2)
    return big.cuda()[..., front:front + h * n].unflatten(-1, (h, n))


@pytest.mark.parametrize("rule", ["scan", "delta"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views_and_strided_pools(rule, dtype):
    """x, B and C as slices of wider rows, the pool as one layer of layer-major and of slot-major pools:
    bit for bit the contiguous call."""
    d = ref.make(3, 37, 4, 32, 64, 2, 15, dtype, rule, "ragged")
    y, g = tree(d), up(d)
    x, B, C = wide(d["x"], 24), wide(d["B"], 8, 16), wide(d["C"], 40, 8)
    S = d["pool"].shape[0]
    major = torch.full((3, S, 4, 32, 64), float("nan"), device="cuda")
    major[1] = g["pool"]
    inner = torch.full((S, 3, 4, 32, 64), float("nan"), device="cuda")
    inner[:, 2] = g["pool"]
    for pool in (major[1], inner[:, 2]):
        got = ssd.tree_step(x, g["dt"], g["A"], B, C, g["parents"], pool, g["slots"], D=g["D"], beta=g["beta"])
        assert torch.equal(got, y)


def test_rows_share_a_slot():
    """Several rows may read one slot (drafts of several samples over one prompt)."""
    d = ref.make(4, 20, 2, 32, 32, 1, 17)
    d["slots"][:] = d["slots"][0].item()
    check_tree(d, "shared slot")


def test_many_rows_fill_the_gpu_like_few():
    """A row's result does not depend on how many rows there are."""
    d = ref.make(40, 30, 16, 64, 128, 2, 19, "bf16", "delta", "ragged")
    y = tree(d)
    for i in (0, 17, 39):
        one = {k: (v[i:i + 1].contiguous() if k in ("x", "dt", "B", "C", "beta", "parents", "slots") else v) for k, v in d.items()}
        assert torch.equal(tree(one)[0], y[i]), i


@pytest.mark.parametrize("rule", ["scan", "delta"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [16, 32, 64, 128, 256])
def test_every_state_width(N, dtype, rule):
    """Every dstate at each number of node tiles and of panels, over the headdims (16 and 32 leave waves
    without columns, 128 needs a second set)."""
    for i, K in enumerate([2, 15, 16, 31, 32, 47, 48, 64, 65, 127, 129, 193]):
        P = [16, 32, 64, 128][(i + N // 16) % 4]
        check_tree(ref.make(2, K, 3, P, N, 1, 700 + K, dtype, rule, ["tree", "holes"][i % 2]), (N, K, P, rule, dtype))


# b, K, H, P, N, G, dtype, kind: enough rows and heads that a work-group of a long tree takes two heads
LONG = [
    (43, 70, 6, 16, 32, 2, "bf16", "holes"),  # (three heads a group: the last one alone)
    (33, 129, 8, 32, 16, 1, "f32", "deep"),
    (33, 65, 8, 64, 128, 4, "bf16", "ragged"),
    (65, 200, 4, 16, 256, 2, "bf16", "line"),
    (65, 200, 4, 64, 256, 1, "bf16", "deep"),
    (33, 256, 8, 16, 64, 1, "f32", "tree"),
    (65, 100, 4, 32, 256, 1, "f32", "deep"),
    (129, 193, 2, 64, 128, 1, "f32", "star"),
]


@pytest.mark.parametrize("rule", ["scan", "delta"])
@pytest.mark.parametrize("case", LONG, ids=lambda c: "b{}K{}H{}P{}N{}G{}{}{}".format(*c))
def test_long_trees_of_many_rows(case, rule):
    """Rows of a call that fills the GPU: the definition's, and bit for bit those of calls with one row; a
    value that is not finite stays in its branch, head and column."""
    b, K, H, P, N, G, dtype, kind = case
    print(f"[tree] {case} {rule}", flush=True)
    d = ref.make(b, K, H, P, N, G, 500 + K, dtype, rule, kind)
    y = tree(d)
    for i in (0, b // 2, b - 1):
        one = {k: (v[i:i + 1].contiguous() if k in ("x", "dt", "B", "C", "beta", "parents", "slots") and v is not None else v)
               for k, v in d.items()}
        assert torch.equal(check_tree(one, (case, rule, i)), y[i:i + 1]), i
    i, k = b // 2, next(n for n, p in enumerate(ref.paths(d["parents"])[b // 2]) if p is not None)
    for name in ("x", "B", "dt", "beta"):
        if d[name] is None:
            continue
        e = {n: (v.clone() if isinstance(v, torch.Tensor) else v) for n, v in d.items()}
        e[name][(i, k, G - 1 if name == "B" else H - 1) + ((3,) if name in "xB" else ())] = float("nan")
        hit = torch.zeros(d["x"].shape, dtype=torch.bool)
        hit[i, below(d, i, k), slice(H - H // G if name == "B" else H - 1, H), 3 if name == "x" else slice(None)] = True
        z = tree(e).cpu()
        assert torch.equal(z[~hit], y.cpu()[~hit]) and not torch.isfinite(z[hit]).any(), name


# ---- commit ----
def commit(d, last, inplace=None):
    g = up(d)
    ssd.tree_commit(g["x"], g["dt"], g["A"], g["B"], g["parents"], torch.tensor(last, dtype=torch.int32, device="cuda"),
                    g["pool"], g["slots"], beta=g["beta"], out_slots=g["out_slots"])
    torch.cuda.synchronize()
    return g["pool"].cpu()


def check_state(got, want, before, tokens, where):
    """Slots that no row writes keep their bits; the others are within STATE per token."""
    touched = (want != before.double()).flatten(1).any(1)
    assert torch.equal(got[~touched].view(torch.int32), before[~touched].view(torch.int32)), where
    scale = max(want.abs().max().item(), before.abs().max().item())
    assert ((got.double() - want).abs() <= STATE * max(1, tokens) * scale).all(), where


@pytest.mark.parametrize("rule", ["scan", "delta"])
@pytest.mark.parametrize("out", [False, True], ids=["inplace", "out"])
@pytest.mark.parametrize("case", [c for c in TREES if c[1] <= 130] + [(1, 256, 1, 16, 32, 1, "bf16", "line")],
                         ids=lambda c: "b{}K{}H{}P{}N{}G{}{}{}".format(*c))
def test_commit_matches_definition(case, rule, out):
    b, K, H, P, N, G, dtype, kind = case
    print(f"[commit] {case} {rule} {out}", flush=True)
    d = ref.make(b, K, H, P, N, G, 400 + K, dtype, rule, kind, out=out)
    for last in ([K - 1 - i % K for i in range(b)], [i % K for i in range(b)]):
        want = ref.commit(d, last)
        deep = max([len(p) for row in ref.paths(d["parents"]) for p in row if p is not None] + [1])
        check_state(commit(d, last), want, d["pool"], deep, (case, last))


def test_commit_of_nothing():
    """-1 keeps the state (and moves it to the out slot); no node, an absent one, an idle row and an out
    slot outside the pool write nothing."""
    for out in (False, True):
        d = ref.make(8, 6, 2, 16, 32, 1, 21, "f32", "delta", "line", out=out)
        d["parents"][3, 2] = -2
        d["slots"][4] = -5
        if out:
            d["out_slots"][5] = d["pool"].shape[0]
        for bad in ("dt", "x", "B", "beta"):
            d[bad][3, 2:] = float("nan")
        last = [-1, 6, -2, 4, 3, 2, 2 ** 31 - 1, 1]
        want = ref.commit(d, last)
        got = commit(d, last)
        check_state(got, want, d["pool"], 6, out)
        if out:
            assert torch.equal(got[d["out_slots"][0]], d["pool"][d["slots"][0]])
            assert torch.equal(got[d["out_slots"][3]], d["pool"][d["out_slots"][3]])


def test_commit_is_the_step_over_the_path():
    """Bit for bit: both are the recurrence in float32."""
    for rule in ("scan", "delta"):
        d = ref.make(1, 40, 4, 64, 128, 2, 23, "bf16", rule, "tree")
        k = max(range(40), key=lambda k: len(ref.paths(d["parents"])[0][k]))
        path = ref.paths(d["parents"])[0][k]
        g = up({n: (d[n][:, path].contiguous() if n in ("x", "dt", "B", "C", "beta") and d[n] is not None else d[n]) for n in d})
        ssd.pool_step(g["x"], g["dt"], g["A"], g["B"], g["C"], g["pool"], g["slots"], D=g["D"], beta=g["beta"])
        assert torch.equal(g["pool"].cpu(), commit(d, [k]))
