"""Trees of so many rows and heads that one launch would have 2^32 threads or more, past which a launch covers
only their remainder and reports nothing: the launches that the entry point makes instead, on the host."""
import ctypes

import pytest

import launch_record as lr
import ssd_chunked_scan_03_amd as ssd


class Args(ctypes.Structure):
    """The kernels' argument (csrc/pool.hpp)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("b", "T")] + [(n, ctypes.c_int) for n in "HPNG"] + \
        [(n, ctypes.c_int64) for n in ("xs", "bs", "cs", "S", "ss")] + \
        [(n, ctypes.c_uint64) for n in ("x", "dt", "A", "B", "C", "D", "beta", "parents", "last", "pool", "slots", "out", "y")]


# rows, nodes, heads, headdim, dstate, groups
BIG = [(65537, 1, 128, 128, 16, 128), (65537, 65, 128, 16, 16, 128), ((1 << 24) - 1, 1, 1, 128, 16, 1),
       ((1 << 24) - 1, 70, 1, 16, 16, 1), (131071, 256, 64, 128, 16, 64), (15, 64, 1 << 20, 16, 16, 1 << 20),
       ((1 << 24) - 1, 1, 1, 64, 16, 1), (65537, 65, 128, 16, 16, 64), (3, 20, 4, 64, 64, 2), (1, 256, 2, 128, 16, 1)]


@pytest.mark.parametrize("rule", ["scan", "delta"])
@pytest.mark.parametrize("dtype", [ssd.SSD_BF16, ssd.SSD_F32], ids=["bf16", "f32"])
def test_every_row_in_launches_under_two_to_the_32(tmp_path, dtype, rule):
    es, exe = (2 if dtype == ssd.SSD_BF16 else 4), lr.recorder(tmp_path)
    names = "x dt A B C D beta parents pool slots y".split()
    calls = []
    for b, K, H, P, N, G in BIG:
        p = ssd.PoolProblem(b, K, H, P, N, G, H * P + 64, G * N + 32, G * N + 64, 3, H * P * N, dtype, 0)
        at = {n: lr.FAKE + i * lr.FAR for i, n in enumerate(names)}
        at["D" if rule == "delta" else "beta"] = 0
        calls.append(("ssd_tree_step", p, [at[n] for n in names] + [0]))
    for (b, K, H, P, N, G), (_, p, _), (st, launches) in zip(BIG, calls, lr.record(exe, calls, ctypes.sizeof(Args))):
        case, row = (b, K, H, P, N, G), 0
        assert st == 0 and lr.fits(launches), (case, [v[:2] for v in launches])
        each = None  # work-groups of a row
        for grid, group, raw in launches:
            a = Args.from_buffer_copy(raw)
            tok = row * K
            at = {n: lr.FAKE + i * lr.FAR for i, n in enumerate(names)}
            want = dict(x=at["x"] + tok * p.xstride * es, dt=at["dt"] + tok * H * 4, A=at["A"], B=at["B"] + tok * p.bstride * es,
                        C=at["C"] + tok * p.cstride * es, D=at["D"] if rule == "scan" else 0,
                        beta=at["beta"] + tok * H * es if rule == "delta" else 0, parents=at["parents"] + tok * 4, pool=at["pool"],
                        slots=at["slots"] + row * 4, y=at["y"] + tok * H * P * es)
            assert {n: getattr(a, n) for n in want} == want, (case, row)
            assert (a.T, a.H, a.P, a.N, a.G, a.S) == (K, H, P, N, G, 3) and a.b > 0
            assert grid[0] % a.b == 0 and grid[1:] == (1, 1) and each in (None, grid[0] // a.b), (case, row)
            each = grid[0] // a.b
            assert each >= G * max(1, P // 64 if K <= 64 else 1), case
            row += a.b
        assert row == b, case
        assert (len(launches) > 1) == (b * each * group[0] > lr.MOST), case
