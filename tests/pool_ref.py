"""Float64 references of the operators on a pool of states, from their definitions: node by node (a
state per node), token by token, and row by row for the pool's pages; and how far a result may be off.
"""
import math

import torch

B16, F32, TWO = 2.0 ** -8, 2.0 ** -24, 2.0 ** -16  # half a step of bfloat16, of float32, of two bfloat16 terms


def make(b, K, H, P, N, G, seed, dtype="bf16", rule="scan", kind="tree", spare=3, out=False, key="unit", dt_hi=0.1,
         D=True):
    g = torch.Generator().manual_seed(seed)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    ru = lambda *s: torch.rand(*s, generator=g)  # noqa: E731
    unit = lambda v: v / v.norm(dim=-1, keepdim=True)  # noqa: E731
    S = (2 if out else 1) * b + spare
    slot = torch.randperm(S, generator=g).to(torch.int32)
    d = dict(x=rn(b, K, H, P).to(td), dt=dt_hi * (0.1 + 0.9 * ru(b, K, H)), A=-torch.exp(ru(H) * math.log(16.0)))
    B = unit(rn(b, K, G, N))
    if key == "same" and K:
        B = B[:, :1].expand(b, K, G, N).contiguous()
    d.update(B=B.to(td), C=unit(rn(b, K, G, N)).to(td), D=rn(H) if rule == "scan" and D else None,
             beta=ru(b, K, H).to(td) if rule == "delta" else None)
    k = torch.arange(K)
    par = (ru(b, K) * k).long().minimum((k - 1).clamp(min=0))
    if kind == "line":
        par = (k - 1).expand(b, K).clone()
    elif kind == "star":
        par = torch.full((b, K), -1)
    elif kind == "deep":  # mostly lines, with a branch now and then
        par = torch.where(ru(b, K) < 0.8, k - 1, par)
    if K:
        par[:, 0] = -1
    if kind == "ragged":
        par = torch.where(k < (1 + (ru(b, 1) * K).long()), par, -2)
    elif kind == "holes":  # absent nodes anywhere, and trees under the held state beside one another
        u = ru(b, K)
        par = torch.where(u < 0.1, -1, par)
        par = torch.where(u > 0.93, -2, torch.where((u > 0.9) & (u <= 0.93), 3 * K + k, par))
    d["parents"] = par.to(torch.int32)
    d["pool"] = 0.3 * rn(S, H, P, N)
    d["slots"] = slot[:b].contiguous()
    d["out_slots"] = slot[b:2 * b].contiguous() if out else None
    return d


def paths(parents):
    """Every present node's path from the held state, itself last; None for absent nodes."""
    out = []
    for row in parents.tolist():
        got = []
        for k, q in enumerate(row):
            ok = -1 <= q < k and (q < 0 or got[q] is not None)
            got.append(None if not ok else ([] if q < 0 else got[q]) + [k])
        out.append(got)
    return out


def _operands(d):
    f = {k: v.double() for k, v in d.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    rep = d["x"].shape[2] // d["B"].shape[2]
    f["key"] = f["B"].repeat_interleave(rep, 2)
    if d.get("C") is not None:
        f["query"] = f["C"].repeat_interleave(rep, 2)
    f["a"] = torch.exp(f["dt"] * f["A"])
    return f


def _next(f, h, i, k):
    h = h * f["a"][i, k][:, None, None]
    u = f["x"][i, k]
    if "beta" in f:
        u = f["beta"][i, k][:, None] * (u - (h * f["key"][i, k][:, None]).sum(-1))
    return h + u[..., None] * f["key"][i, k][:, None]


def live(d, i, which="slots"):
    s = int(d[which][i])
    return s if 0 <= s < d["pool"].shape[0] else None


def tree(d):
    """y [b, K, H, P] (zero where a node is absent or its row idle)."""
    f = _operands(d)
    y = torch.zeros_like(f["x"])
    for i, got in enumerate(paths(d["parents"])):
        if live(d, i) is None:
            continue
        states = {-1: f["pool"][live(d, i)]}
        for k, path in enumerate(got):
            if path is None:
                continue
            states[k] = _next(f, states[path[-2] if len(path) > 1 else -1], i, k)
            y[i, k] = (states[k] * f["query"][i, k][:, None]).sum(-1)
            if "D" in f:
                y[i, k] += f["D"][:, None] * f["x"][i, k]
    return y


def tree_limit(d, y):
    """How far tree_step's y may be off.  With u the added columns, T_kj = beta_k W_kj (B_k . B_j) and
    ubar the solution of ubar_k = beta (|x| + E |h B|) + sum_j |T_kj| ubar_j (at least |u|):
    * y is rounded once: half a step of its type;
    * float32 sums over n = dstate products, the nodes of the path and the steps of the exponent (s binary
      orders of decay, off by s 2^-24, and 2 for the exponential): n 2^-24 of the absolute terms;
    * bfloat16: the state, T, the inverse of its diagonal blocks, the right side, u and M = W (C . B)
      enter the matrix cores in two terms: 6 2^-16 of the terms that hold them;
    * what u is off by passes on to the nodes below through |T|, and to y through |M|."""
    f = _operands(d)
    half = d["x"].dtype == torch.bfloat16
    N = f["B"].shape[3]
    lim = torch.zeros_like(y)
    for i, got in enumerate(paths(d["parents"])):
        if live(d, i) is None:
            continue
        h = f["pool"][live(d, i)]
        ub, du = {}, {}
        for k, path in enumerate(got):
            if path is None:
                continue
            steps = -f["dt"][i] * f["A"] / math.log(2.0)  # [K, H] binary orders
            tail = torch.zeros_like(steps[0])
            w = {}
            for j in reversed(path):
                w[j] = torch.exp2(-tail)
                tail = tail + steps[j]
            E = torch.exp2(-tail)[:, None]
            few = (N + len(path) + 2 + tail.clamp(max=150).max().item()) * F32
            two = 6 * TWO if half else 6 * F32
            bk, ck = f["key"][i, k], f["query"][i, k]

            def terms(v, to, absolute, own):
                """E |h v| and sum_j W_kj |v . B_j| to_j; absolute: of the products' absolute values."""
                vh = (h.abs() * v.abs()[:, None]).sum(-1) if absolute else (h * v[:, None]).sum(-1).abs()
                s = E * vh
                for j in path if own else path[:-1]:
                    kj = f["key"][i, j]
                    dot = (v.abs() * kj.abs()).sum(-1) if absolute else (v * kj).sum(-1).abs()
                    s = s + w[j][:, None] * dot[:, None] * to[j]
                return s

            if "beta" in f:
                bt = f["beta"][i, k].abs()[:, None]
                ub[k] = bt * (f["x"][i, k].abs() + terms(bk, ub, False, False))
                near = {j: du[j] for j in path[:-1]}
                zero = E * (h * bk[:, None]).sum(-1).abs()
                du[k] = two * (ub[k] + bt * E * (h.abs() * bk.abs()[:, None]).sum(-1)) \
                    + few * bt * terms(bk, ub, True, False) + bt * (terms(bk, near, False, False) - zero)
            else:
                ub[k], du[k] = f["x"][i, k].abs(), torch.zeros_like(f["x"][i, k])
            zero = E * (h * ck[:, None]).sum(-1).abs()
            lim[i, k] = (B16 if half else F32) * y[i, k].abs() + (two + few) * terms(ck, ub, True, True) \
                + terms(ck, du, False, True) - zero
            if "D" in f:
                lim[i, k] += 2 * F32 * (f["D"][:, None] * f["x"][i, k]).abs()
    return lim


def commit(d, last):
    """The pool behind tree_commit."""
    f = _operands(d)
    pool = f["pool"].clone()
    for i, got in enumerate(paths(d["parents"])):
        k = int(last[i])
        if live(d, i) is None or k < -1 or k >= len(got) or (k >= 0 and got[k] is None):
            continue
        h = f["pool"][live(d, i)]
        for j in [] if k < 0 else got[k]:
            h = _next(f, h, i, j)
        to = live(d, i, "slots" if d["out_slots"] is None else "out_slots")
        if to is not None:
            pool[to] = h
    return pool


def step(d):
    """(y, the pool) of pool_step."""
    f = _operands(d)
    pool, y = f["pool"].clone(), torch.zeros_like(f["x"])
    for i in range(y.shape[0]):
        if live(d, i) is None:
            continue
        h = f["pool"][live(d, i)]
        for t in range(y.shape[1]):
            h = _next(f, h, i, t)
            y[i, t] = (h * f["query"][i, t][:, None]).sum(-1)
            if "D" in f:
                y[i, t] += f["D"][:, None] * f["x"][i, t]
        to = live(d, i, "slots" if d["out_slots"] is None else "out_slots")
        if to is not None:
            pool[to] = h
    return y, pool


def fork(pool, table, sources):
    """(new table, pool after the moves) of pool_fork."""
    S, R = pool.shape[-4], table.numel()
    slot = lambda r: int(table[r]) if 0 <= int(table[r]) < S else None  # noqa: E731
    want = [slot(q) if 0 <= q < R else None for q in sources.tolist()]
    owner = {}  # of the rows that go on from a slot: one that had it, else the lowest
    for r in sorted(range(R), key=lambda r: (want[r] is None or slot(r) != want[r], r)):
        if want[r] is not None:
            owner.setdefault(want[r], r)
    free = iter([s for s in range(S) if s not in owner])
    new, after = [], pool.clone()
    for r, s in enumerate(want):
        if s is not None and owner[s] == r:
            new.append(s)
        elif s is not None or int(sources[r]) == -2:
            new.append(next(free))
            after[..., new[-1], :, :, :] = 0.0 if s is None else pool[..., s, :, :, :]
        else:
            new.append(-1)
    return torch.tensor(new, dtype=torch.int32), after


def compact(pool, table):
    """(new table, count, pool) of pool_compact."""
    S = pool.shape[-4]
    named = sorted({s for s in table.tolist() if 0 <= s < S})
    n = len(named)
    moved = dict(zip([s for s in named if s >= n], sorted(set(range(n)) - set(named))))
    after = pool.clone()
    for s, t in moved.items():
        after[..., t, :, :, :] = pool[..., s, :, :, :]
    new = [moved.get(s, s) if 0 <= s < S else -1 for s in table.tolist()]
    return torch.tensor(new, dtype=torch.int32), n, after
