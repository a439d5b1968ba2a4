"""The operators on a pool of states at the far ends of their ranges."""
import pytest
import torch

import pool_ref as ref
import ssd_chunked_scan_03_amd as ssd
from test_gpu_tree import check_state, check_tree, commit, tree, up

pytestmark = pytest.mark.gpu


# b, K, H, P, N, G, rule: 4 295 032 832 threads each in one launch
@pytest.mark.parametrize("case", [(65537, 1, 128, 128, 16, 128, "scan"), (65537, 1, 128, 128, 16, 128, "delta"),
                                  (65537, 65, 128, 16, 16, 128, "scan")], ids=lambda c: "b{}K{}H{}P{}N{}G{}{}".format(*c))
def test_trees_of_more_threads_than_a_launch(case):
    """Every row is written, and rows at the ends and around the launches' border are a small call's bits."""
    b, K, H, P, N, G, rule = case
    print(f"[far] {case}", flush=True)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(91)
    x, B, C = (torch.empty(b, K, n, m, **bf).normal_(generator=g) for n, m in ((H, P), (G, N), (G, N)))
    B, C = B.mul_(0.25), C.mul_(0.25)
    dt = 0.1 * torch.rand(b, K, H, generator=g, device="cuda")
    A = -1 - 15 * torch.rand(H, generator=g, device="cuda")
    beta = torch.rand(b, K, H, generator=g, device="cuda").bfloat16() if rule == "delta" else None
    D = torch.randn(H, generator=g, device="cuda") if rule == "scan" else None
    pool = torch.randn(5, H, P, N, generator=g, device="cuda")
    slots = torch.randint(0, 5, (b,), generator=g, device="cuda", dtype=torch.int32)
    parents = (torch.rand(b, K, generator=g, device="cuda") * torch.arange(K, device="cuda")).int() - 1
    y = torch.full((b, K, H, P), float("nan"), **bf)
    prob = ssd.PoolProblem(b, K, H, P, N, G, H * P, G * N, G * N, 5, H * P * N, ssd.SSD_BF16, 0)
    ssd.tree_step_into(prob, x, dt, A, B, C, D, beta, parents, pool, slots, y)
    torch.cuda.synchronize()
    for lo in range(0, b, 4096):
        assert torch.isfinite(y[lo:lo + 4096]).all(), lo
    most = 0xffffffff // (H * max(1, P // 64 if K <= 64 else 1) * (256 if K <= 64 else 512))
    for lo in (0, most - 2, most, b - 3):
        s = slice(lo, min(b, lo + 3))
        one = ssd.tree_step(x[s], dt[s], A, B[s], C[s], parents[s], pool, slots[s], D=D, beta=None if beta is None else beta[s])
        assert torch.equal(one, y[s]), lo


# K: every number of node tiles, and panels
@pytest.mark.parametrize("K", [1, 16, 17, 48, 64, 65, 200])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_row_of_b_whose_square_leaves_float32(K, dtype):
    """The delta rule at a leaf with a finite B of norm 8e19: |B|^2 is in none of its formulas, so its y is the
    definition's, and every other node keeps its bits."""
    d = ref.make(2, K, 4, 32, 64, 2, 95, dtype, "delta", "tree")
    clean = tree(d)
    sign = 1 - 2 * (torch.arange(64) % 3 == 1).float()
    d["B"][1, K - 1, 1] = (1e19 * sign).to(d["B"].dtype)
    d["C"][1, K - 1, 1] *= 1e-19
    assert (d["B"][1, K - 1, 1].double() ** 2).sum() > torch.finfo(torch.float32).max
    y = check_tree(d, (K, dtype))
    hit = torch.zeros(y.shape, dtype=torch.bool)
    hit[1, K - 1, 2:] = True
    assert torch.equal(y.cpu()[~hit], clean.cpu()[~hit])


# b, K, H, P, N, G, dtype, kind
SAME = [(32, 40, 32, 128, 128, 16, "bf16", "tree"), (16, 200, 32, 64, 256, 8, "bf16", "line"), (64, 64, 16, 64, 128, 1, "bf16", "tree"),
        (33, 129, 8, 32, 64, 2, "f32", "deep"), (20, 27, 6, 32, 64, 3, "f32", "ragged")]


@pytest.mark.parametrize("rule", ["scan", "delta"])
@pytest.mark.parametrize("case", SAME, ids=lambda c: "b{}K{}H{}P{}N{}G{}{}{}".format(*c))
def test_the_same_tree_is_the_same_bits(case, rule):
    """Calls on the same inputs, back to back and beside other work on another stream."""
    b, K, H, P, N, G, dtype, kind = case
    d = up(ref.make(b, K, H, P, N, G, 93, dtype, rule, kind))
    call = lambda: ssd.tree_step(d["x"], d["dt"], d["A"], d["B"], d["C"], d["parents"], d["pool"], d["slots"], D=d["D"], beta=d["beta"])  # noqa: E731
    y = call()
    assert all(torch.equal(call(), y) for _ in range(20))
    side, big = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(10):
            big = big @ big * 1e-3
    again = [call() for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(v, y) for v in again)


@pytest.mark.parametrize("rule", ["scan", "delta"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [20, 80])
def test_an_infinite_step_forgets(K, dtype, rule):
    """dt = inf decays by exp(-inf) = 0, a value like any other: at and below such nodes y and the committed
    states are the definition's, and elsewhere the bits of the call without them."""
    d = ref.make(2, K, 4, 32, 64, 2, 97, dtype, rule, "deep")
    clean = tree(d)
    d["dt"][1, K // 3, 2] = d["dt"][1, K - 2, 0] = float("inf")
    y = check_tree(d, (K, dtype, rule))
    hit = torch.zeros(y.shape, dtype=torch.bool)
    for k, h in ((K // 3, 2), (K - 2, 0)):
        hit[1, [n for n, path in enumerate(ref.paths(d["parents"])[1]) if k in path], h] = True
    assert hit.any() and torch.equal(y.cpu()[~hit], clean.cpu()[~hit]) and not torch.equal(y.cpu(), clean.cpu())
    last = [K - 1, K // 3]
    deep = max(len(path) for row in ref.paths(d["parents"]) for path in row)
    check_state(commit(d, last), ref.commit(d, last), d["pool"], deep, (K, dtype, rule))
