"""GPU parity of the decode step through slots and of the pool's pages, and runs of the pool's operators
together: a served loop with drafts, graphs, streams, slots past 32-bit offsets."""
import pytest
import torch

import pool_ref as ref
import ssd_chunked_scan_03_amd as ssd
from test_gpu_tree import STATE, check_state, up, wide

pytestmark = pytest.mark.gpu


def step(g):
    return ssd.pool_step(g["x"], g["dt"], g["A"], g["B"], g["C"], g["pool"], g["slots"], D=g["D"], beta=g["beta"],
                         out_slots=g["out_slots"])


def check_y(got, want, scale, tokens, dtype, where):
    """y is a sum over dstate of the state, rounded once: STATE of the largest value per token, and half a step."""
    half = ref.B16 if dtype == "bf16" else ref.F32
    assert ((got.double().cpu() - want).abs() <= half * want.abs() + STATE * (tokens + 1) * scale).all(), where


# b, T, H, P, N, G, dtype
STEPS = [(1, 1, 1, 16, 16, 1, "bf16"), (3, 1, 4, 128, 128, 2, "bf16"), (2, 5, 3, 32, 64, 3, "f32"),
         (4, 1, 2, 64, 256, 1, "bf16"), (1, 9, 2, 128, 32, 2, "f32"), (5, 2, 48, 64, 128, 1, "bf16")]


@pytest.mark.parametrize("rule", ["scan", "delta"])
@pytest.mark.parametrize("out", [False, True], ids=["inplace", "out"])
@pytest.mark.parametrize("case", STEPS, ids=lambda c: "b{}T{}H{}P{}N{}G{}{}".format(*c))
def test_step_matches_definition(case, rule, out):
    b, T, H, P, N, G, dtype = case
    print(f"[pool step] {case} {rule} {out}", flush=True)
    d = ref.make(b, T, H, P, N, G, 500 + T, dtype, rule, out=out)
    g = up(d)
    y = step(g)
    want, pool = ref.step(d)
    check_y(y, want, max(pool.abs().max().item(), want.abs().max().item(), 1.0), T, dtype, case)
    check_state(g["pool"].cpu(), pool, d["pool"], T, case)


@pytest.mark.parametrize("rule", ["scan", "delta"])
def test_step_is_the_held_state_step(rule):
    """Through slots or on a contiguous batch: the same recurrence."""
    d = ref.make(3, 4, 4, 64, 128, 2, 31, "bf16", rule)
    g = up(d)
    h = g["pool"][g["slots"].long()].contiguous()
    y = step(g)
    if rule == "scan":
        other = ssd.step(g["x"], g["dt"], g["A"], g["B"], g["C"], h, g["D"])
    else:
        other = ssd.delta_step(g["x"], g["dt"], g["A"], g["B"], g["C"], g["beta"], h)
    scale = max(h.abs().max().item(), y.abs().max().item(), 1.0)
    assert (y.double() - other.double()).abs().max().item() <= 2 * ref.B16 * scale
    assert (g["pool"][g["slots"].long()] - h).abs().max().item() <= 2 * 4 * STATE * scale


def test_step_idle_rows_shared_slots_and_views():
    """Idle rows are zero and touch nothing, an out slot outside the pool leaves no state, rows that share
    a slot write their own; views give the same bits."""
    d = ref.make(6, 3, 2, 32, 64, 1, 33, "bf16", "delta", out=True)
    d["slots"][1], d["slots"][2] = -1, d["pool"].shape[0]
    d["slots"][4] = d["slots"][3].item()
    d["out_slots"][5] = -7
    for name in ("x", "B", "C", "dt", "beta"):
        d[name][1:3] = float("nan")
    g = up(d)
    y = step(g)
    d0 = {k: (torch.nan_to_num(v) if isinstance(v, torch.Tensor) and v.is_floating_point() else v) for k, v in d.items()}
    want, pool = ref.step(d0)
    assert not y[1:3].any()
    check_y(y, want, 2.0, 3, "bf16", "idle")
    check_state(g["pool"].cpu(), pool, d["pool"], 3, "idle")
    after = g["pool"].clone()
    g = up(d)
    g.update(x=wide(d["x"], 8), B=wide(d["B"], 16, 8), C=wide(d["C"], 0, 24))
    inner = torch.zeros(d["pool"].shape[0], 2, *d["pool"].shape[1:], device="cuda")
    inner[:, 1] = g["pool"]
    g["pool"] = inner[:, 1]
    again = step(g)
    assert torch.equal(again, y) and torch.equal(inner[:, 1], after) and not inner[:, 0].any()


def test_no_tokens():
    """Without tokens a state goes to its out slot, and in place nothing happens."""
    d = ref.make(2, 0, 2, 16, 16, 1, 35, "bf16", "scan", out=True)
    g = up(d)
    assert step(g).shape == (2, 0, 2, 16)
    assert torch.equal(g["pool"][g["out_slots"].long()].cpu(), d["pool"][d["slots"].long()])
    g = up(dict(d, out_slots=None))
    step(g)
    assert torch.equal(g["pool"].cpu(), d["pool"])
    last = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    g = up(d)
    ssd.tree_commit(g["x"], g["dt"], g["A"], g["B"], g["parents"], last, g["pool"], g["slots"], out_slots=g["out_slots"])
    assert torch.equal(g["pool"][g["out_slots"].long()].cpu(), d["pool"][d["slots"].long()])
    assert ssd.tree_step(g["x"], g["dt"], g["A"], g["B"], g["C"], g["parents"], g["pool"], g["slots"]).numel() == 0


# ---- pages ----
def page_case(seed, layers, S, R, shape, inner=False):
    """A pool, a table (some rows empty, some sharing a slot, some entries no slot) and sources of every kind."""
    g = torch.Generator().manual_seed(seed)
    pool = torch.randn(layers, S, *shape, generator=g)
    table = torch.randperm(max(S, 1), generator=g)[:R].to(torch.int32) if S else torch.zeros(0, dtype=torch.int32)
    sources = torch.randint(0, max(R, 1), (R,), generator=g).to(torch.int32)
    for r in range(R):
        u = torch.rand(3, generator=g)
        if u[0] < 0.1:
            table[r] = [-1, -9, S, 2 ** 31 - 1][int(u[1] * 4)]
        elif u[0] < 0.2:
            table[r] = table[int(u[1] * R)]
        if u[2] < 0.2:
            sources[r] = [-1, -2, -2, R, -3][int(u[1] * 5)]
        elif u[2] < 0.5:
            sources[r] = r
    dev = pool.cuda()
    if inner:
        dev = dev.transpose(0, 1).contiguous().transpose(0, 1)  # slots of whole layers
    return pool, dev, table, sources


PAGES = [(1, 1, 1, (1, 16, 16)), (1, 5, 3, (2, 16, 16)), (3, 9, 9, (2, 16, 32)), (2, 64, 60, (1, 32, 32)),
         (4, 65, 65, (3, 16, 16)), (1, 130, 100, (5, 64, 128)), (2, 700, 600, (1, 16, 16)), (1, 7, 0, (1, 16, 16)),
         (0, 4, 3, (1, 16, 16)), (1, 16384, 16384, (1, 16, 16)), (1, 16384, 300, (1, 16, 16)), (25, 33, 20, (7, 16, 64))]


@pytest.mark.parametrize("inner", [False, True], ids=["layers", "slots"])
@pytest.mark.parametrize("case", PAGES, ids=lambda c: "L{}S{}R{}".format(*c[:3]))
def test_fork_and_compact_match_definition(case, inner):
    layers, S, R, shape = case
    print(f"[pages] {case} {inner}", flush=True)
    for seed in range(1 if S > 5000 else 3):
        pool, dev, table, sources = page_case(600 + seed, layers, S, R, shape, inner)
        want, after = ref.fork(pool, table, sources)
        new = ssd.pool_fork(dev, table.cuda(), sources.cuda())
        torch.cuda.synchronize()
        assert torch.equal(new.cpu(), want) and torch.equal(dev.cpu(), after)
        named = want[want >= 0]
        assert len(set(named.tolist())) == named.numel()
        pool, dev, table, _ = page_case(700 + seed, layers, S, R, shape, inner)
        want, n, after = ref.compact(pool, table)
        new, count = ssd.pool_compact(dev, table.cuda())
        torch.cuda.synchronize()
        assert torch.equal(new.cpu(), want) and count.tolist() == [n] and torch.equal(dev.cpu(), after)


def test_one_layer_pool_and_strided_slots():
    """A [S, H, P, N] pool, and slots with room between them that stays as it is."""
    big = torch.randn(9, 3, 2, 16, 16, device="cuda")
    keep, pool = big.clone(), big[:, 1]
    table = torch.tensor([7, 2, 5], dtype=torch.int32)
    sources = torch.tensor([0, 0, -2], dtype=torch.int32)
    want, after = ref.fork(pool.cpu(), table, sources)
    new = ssd.pool_fork(pool, table.cuda(), sources.cuda())
    assert torch.equal(new.cpu(), want) and torch.equal(pool.cpu(), after)
    assert torch.equal(big[:, 0], keep[:, 0]) and torch.equal(big[:, 2], keep[:, 2])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -0.0])
def test_pages_move_bits(bad):
    pool = torch.full((1, 4, 1, 16, 16), bad, device="cuda")
    pool[0, 3].view(torch.int32)[...] = torch.arange(256, device="cuda", dtype=torch.int32).view(1, 16, 16) + 0x7f800001
    table = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    new = ssd.pool_fork(pool, table, torch.tensor([0, 0], dtype=torch.int32, device="cuda"))
    assert new.tolist() == [3, 0]
    assert torch.equal(pool[0, 0].view(torch.int32), pool[0, 3].view(torch.int32))


# ---- together ----
def take(g, lo, hi, names=("x", "dt", "B", "C", "beta")):
    return {k: (v[:, lo:hi].contiguous() if k in names and v is not None else v) for k, v in g.items()}


@pytest.mark.parametrize("rule", ["scan", "delta"])
def test_served_loop_with_drafts(rule):
    """Prompts through the packed forward into slots; a fork into samples; rounds of drafted trees, each
    committed; an ended row, a compaction, and a decode step: against the definition's recurrence."""
    H, P, N, G, L = 4, 64, 64, 2, 2
    rows, S = 6, 9
    lens = [70, 3, 129]
    gen = torch.Generator().manual_seed(41)
    td = torch.bfloat16
    pool = torch.randn(L, S, H, P, N, generator=gen).cuda()
    states = {}  # row -> per layer the float64 state
    table = torch.tensor([4, 8, 2, -1, -1, -1], dtype=torch.int32, device="cuda")
    new = ssd.pool_fork(pool, table, torch.tensor([-2, -2, -2, -1, -1, -1], dtype=torch.int32, device="cuda"))
    layers = []
    for l in range(L):
        d = ref.make(1, sum(lens), H, P, N, G, 50 + l, "bf16", rule, "line", spare=0)
        g = up(d)
        cu = torch.tensor([0, 70, 73, 202], dtype=torch.int32, device="cuda")
        at = new[:3].long()
        flat = {k: g[k][0] for k in ("x", "dt", "B", "C")}
        args = (flat["x"], flat["dt"], g["A"], flat["B"], flat["C"])
        h0 = pool[l][at].contiguous()
        assert not h0.any()
        if rule == "scan":
            _, hT = ssd.scan_fwd_varlen(*args, cu, g["D"], h0)
        else:
            _, hT = ssd.delta_fwd_varlen(*args, g["beta"][0], cu, h0)
        pool[l][at] = hT
        layers.append(d)
        lo = 0
        for r, n in enumerate(lens):
            one = take(d, lo, lo + n)
            one.update(pool=torch.zeros(1, H, P, N), slots=torch.zeros(1, dtype=torch.int32), out_slots=None)
            states.setdefault(r, []).append(ref.step(one)[1][0])
            lo += n
    # samples: row 0's prompt also in rows 3 and 4, row 2's in row 5
    table = ssd.pool_fork(pool, new, torch.tensor([0, 1, 2, 0, 0, 2], dtype=torch.int32, device="cuda"))
    for r, s in ((3, 0), (4, 0), (5, 2)):
        states[r] = [v.clone() for v in states[s]]
    order = list(range(rows))
    for turn, kind in enumerate(("tree", "ragged", "line")):
        parents = ref.make(rows, 9, H, P, N, G, 70 + turn, "bf16", rule, kind)["parents"]
        present = [[k for k, p in enumerate(row) if p is not None] for row in ref.paths(parents)]
        last = [-1 if r == 4 else present[r][-1] for r in range(rows)]
        for l in range(L):
            d = ref.make(rows, 9, H, P, N, G, 80 + 10 * turn + l, "bf16", rule, kind)
            d.update(A=layers[l]["A"], D=layers[l]["D"], parents=parents, slots=torch.arange(rows, dtype=torch.int32),
                     pool=torch.stack([states[r][l] for r in range(rows)]))
            g = up(d)
            y = ssd.tree_step(g["x"], g["dt"], g["A"], g["B"], g["C"], g["parents"], pool[l], table, D=g["D"], beta=g["beta"])
            want = ref.tree(d)
            assert ((y.double().cpu() - want).abs() <= 2e-2 * want.abs().max()).all()
            ssd.tree_commit(g["x"], g["dt"], g["A"], g["B"], g["parents"], torch.tensor(last, dtype=torch.int32, device="cuda"),
                            pool[l], table, beta=g["beta"])
            after = ref.commit(d, last)
            for r in range(rows):
                states[r][l] = after[r]
    # row 1 ends; the rest comes together at the front
    table = ssd.pool_fork(pool, table, torch.tensor([0, -1, 2, 3, 4, 5], dtype=torch.int32, device="cuda"))
    table, count = ssd.pool_compact(pool, table)
    assert count.tolist() == [5] and sorted(table.tolist()) == [-1, 0, 1, 2, 3, 4] and table[1].item() == -1
    for l in range(L):
        d = ref.make(rows, 1, H, P, N, G, 120 + l, "bf16", rule)
        live = [r for r in order if r != 1]
        d.update(A=layers[l]["A"], D=layers[l]["D"], slots=torch.arange(rows, dtype=torch.int32), out_slots=None,
                 pool=torch.stack([states[r][l] for r in order]))
        g = up(d)
        y = ssd.pool_step(g["x"], g["dt"], g["A"], g["B"], g["C"], pool[l], table, D=g["D"], beta=g["beta"])
        want, after = ref.step(d)
        assert not y[1].any()
        assert ((y.double().cpu() - want)[live].abs() <= 2e-2 * want.abs().max()).all()
        got = pool[l][table.long()].double().cpu()
        assert ((got - after)[live].abs() <= 2e-2 * after.abs().max()).all()


def graph_of(run):
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


@pytest.mark.parametrize("rule", ["scan", "delta"])
def test_graphs_follow_their_tensors(rule):
    """A captured round (draft, commit, fork, compact, step) replayed with other tables, trees and states
    in the captured tensors, eager work between: every replay is the eager round's bits."""
    H, P, N, G, b, K, S = 4, 64, 128, 2, 5, 33, 8
    mk = lambda seed: up(ref.make(b, K, H, P, N, G, seed, "bf16", rule, "ragged", spare=S - b))  # noqa: E731
    t = mk(1)
    t["last"] = torch.zeros(b, dtype=torch.int32, device="cuda")
    t["sources"] = torch.zeros(b, dtype=torch.int32, device="cuda")
    y, y1 = torch.empty_like(t["x"]), torch.empty_like(t["x"][:, :1].contiguous())
    new, packed, count = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (b, b, 1))
    one = take(t, 0, 1)
    prob = ssd.PoolProblem(b, K, H, P, N, G, H * P, G * N, G * N, S, H * P * N, ssd.SSD_BF16, 0)
    single = ssd.PoolProblem(b, 1, H, P, N, G, H * P, G * N, G * N, S, H * P * N, ssd.SSD_BF16, 0)
    pages = ssd.Pages(b, 1, S, H * P * N, 0, H * P * N)

    def run():
        ssd.tree_step_into(prob, t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], t["beta"], t["parents"], t["pool"], t["slots"], y)
        ssd.tree_commit_into(prob, t["x"], t["dt"], t["A"], t["B"], t["beta"], t["parents"], t["last"], t["pool"], t["slots"], None)
        ssd.pool_fork_into(pages, t["pool"], t["slots"], t["sources"], new)
        ssd.pool_compact_into(pages, t["pool"], new, packed, count)
        ssd.pool_step_into(single, one["x"], one["dt"], t["A"], one["B"], one["C"], t["D"], one["beta"], t["pool"], packed, None, y1)

    g = graph_of(run)
    for seed in (2, 3, 4, 5):
        n = mk(seed)
        for k in ("x", "dt", "B", "C", "beta", "parents", "pool", "slots", "A"):
            if n[k] is not None:
                t[k].copy_(n[k])
        t["last"].copy_(torch.arange(b) % 3 - 1)
        t["sources"].copy_(torch.randint(-2, b, (b,), generator=torch.Generator().manual_seed(seed)))
        before = t["pool"].clone()
        run()
        torch.cuda.synchronize()
        want = [v.clone() for v in (y, t["pool"], new, packed, count, y1)]
        t["pool"].copy_(before)
        for v in (y, y1):
            v.fill_(float("nan"))
        for v in (new, packed, count):
            v.fill_(-77)
        float((torch.randn(1 << 20, device="cuda") ** 2).sum())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for got, w in zip((y, t["pool"], new, packed, count, y1), want):
            assert torch.equal(got, w), seed


@pytest.mark.parametrize("rule", ["scan", "delta"])
def test_long_trees_captured_and_as_views(rule):
    """Trees of several panels, two heads a work-group: x, B and C out of wider rows and a layer of a slot-major
    pool are the contiguous call's bits, and so is every replay of a captured call on other values."""
    b, K, H, P, N, G, S = 33, 150, 8, 32, 64, 2, 36
    d = ref.make(b, K, H, P, N, G, 61, "bf16", rule, "holes", spare=S - b)
    g = up(d)
    y = torch.empty_like(g["x"])
    prob = ssd.PoolProblem(b, K, H, P, N, G, H * P, G * N, G * N, S, H * P * N, ssd.SSD_BF16, 0)

    def run():
        ssd.tree_step_into(prob, g["x"], g["dt"], g["A"], g["B"], g["C"], g["D"], g["beta"], g["parents"], g["pool"], g["slots"], y)

    run()
    inner = torch.full((S, 3, H, P, N), float("nan"), device="cuda")
    inner[:, 1] = g["pool"]
    got = ssd.tree_step(wide(d["x"], 24), g["dt"], g["A"], wide(d["B"], 8, 16), wide(d["C"], 40, 8), g["parents"], inner[:, 1],
                        g["slots"], D=g["D"], beta=g["beta"])
    assert torch.equal(got, y)
    graph = graph_of(run)
    for seed in (62, 63, 64):
        n = up(ref.make(b, K, H, P, N, G, seed, "bf16", rule, ["deep", "ragged", "tree"][seed - 62], spare=S - b))
        for k in ("x", "dt", "B", "C", "D", "beta", "parents", "pool", "slots", "A"):
            if n[k] is not None:
                g[k].copy_(n[k])
        run()
        torch.cuda.synchronize()
        want = y.clone()
        y.fill_(float("nan"))
        float((torch.randn(1 << 20, device="cuda") ** 2).sum())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), seed


def test_calls_on_another_stream():
    """Work goes to the current stream, in order with what it follows there."""
    d = ref.make(4, 20, 4, 64, 128, 2, 45, "bf16", "delta", "tree", out=True)
    g = up(d)
    args = lambda g: (g["x"], g["dt"], g["A"], g["B"], g["C"])  # noqa: E731
    y = ssd.tree_step(*args(g), g["parents"], g["pool"], g["slots"], beta=g["beta"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        late = {k: (torch.zeros_like(v) if isinstance(v, torch.Tensor) else v) for k, v in g.items()}
        torch.randn(4096, 4096, device="cuda") @ torch.randn(4096, 4096, device="cuda")
        for k, v in g.items():
            if isinstance(v, torch.Tensor):
                late[k].copy_(v)
        got = ssd.tree_step(*args(late), late["parents"], late["pool"], late["slots"], beta=late["beta"])
    s.synchronize()
    assert torch.equal(got, y)


def test_slots_past_32_bit_offsets():
    """The last slots of a 10 GB pool: their elements lie past 2^31."""
    H, P, N, S = 64, 128, 256, 1200
    assert (S - 2) * H * P * N > 2 ** 31
    d = ref.make(2, 4, H, P, N, 1, 47, "bf16", "delta", "tree", spare=0)
    pool = torch.empty(S, H, P, N, device="cuda")
    pool[-2:] = d["pool"].cuda()
    g = up(dict(d, pool=None, slots=torch.tensor([S - 1, S - 2], dtype=torch.int32)))
    e = dict(d, slots=torch.tensor([1, 0], dtype=torch.int32))
    y = ssd.tree_step(g["x"], g["dt"], g["A"], g["B"], g["C"], g["parents"], pool, g["slots"], beta=g["beta"])
    h = up(e)
    assert torch.equal(y, ssd.tree_step(h["x"], h["dt"], h["A"], h["B"], h["C"], h["parents"], h["pool"], h["slots"], beta=h["beta"]))
    last = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    ssd.tree_commit(g["x"], g["dt"], g["A"], g["B"], g["parents"], last, pool, g["slots"], beta=g["beta"])
    ssd.tree_commit(h["x"], h["dt"], h["A"], h["B"], h["parents"], last, h["pool"], h["slots"], beta=h["beta"])
    assert torch.equal(pool[-2:], h["pool"])
    table, count = ssd.pool_compact(pool, g["slots"])
    assert table.tolist() == [1, 0] and count.tolist() == [2]
    assert torch.equal(pool[:2], h["pool"])
