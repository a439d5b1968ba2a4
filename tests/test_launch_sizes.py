"""Every entry point at sizes around the most threads that a launch may have, on the host: a call is refused before
anything is enqueued, or each of its launches stays under 2^32 threads along every dimension of its grid.  (Past
that a launch covers only the remainder and reports nothing.)"""
import ctypes
import random

import pytest

import launch_record as lr
import ssd_chunked_scan_03_amd as ssd

UNSUPPORTED = 3
# entry point: its operands, its workspace's query and what that takes beside the problem
SCAN = {
    "ssd_scan_fwd": (9, "ssd_workspace_bytes", 0), "ssd_diag_scan_fwd": (9, "ssd_workspace_bytes", 1),
    "ssd_scan_fwd_varlen": (10, "ssd_varlen_workspace_bytes"), "ssd_step": (8, None), "ssd_diag_step": (8, None),
    "ssd_scan_bwd": (16, "ssd_bwd_workspace_bytes"), "ssd_diag_scan_bwd": (16, "ssd_diag_bwd_workspace_bytes"),
    "ssd_delta_fwd": (9, "ssd_delta_workspace_bytes"), "ssd_delta_fwd_varlen": (10, "ssd_delta_varlen_workspace_bytes"),
    "ssd_delta_step": (8, None), "ssd_delta_bwd": (16, "ssd_delta_bwd_workspace_bytes"),
}


def scan_call(name, b, T, H, P, N, G, Q, dtype):
    """None where an operand would be wider than the operands' distance."""
    n, workspace, *more = SCAN[name]
    p = ssd.make_problem(b, T, H, P, N, G, Q, dtype)
    es = 2 if dtype == ssd.SSD_BF16 else 4
    ws = [] if workspace is None else [lr.FAKE + 30 * lr.FAR, int(getattr(ssd._load(), workspace)(ctypes.byref(p), *more))]
    if max([b * T * H * P * es, b * T * G * N * es, b * H * P * N * 4] + ws[1:]) >= lr.FAR:
        return None
    return name, p, [lr.FAKE + i * lr.FAR for i in range(n)] + ws + [0]


def check(tmp_path, calls):
    states = []
    for call, (st, launches) in zip(calls, lr.record(lr.recorder(tmp_path), calls)):
        what = call[0], [(f, getattr(call[1], f)) for f, _ in call[1]._fields_]
        assert st in (0, UNSUPPORTED), (what, st)
        assert lr.fits(launches) and (st == 0 or not launches), (what, st, [v[:2] for v in launches])
        states.append(st)
    return states


@pytest.mark.parametrize("name", list(SCAN))
def test_scan_and_delta_rule(tmp_path, name):
    rng, calls = random.Random(name), []
    while len(calls) < 1500:
        P, N = rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128, 256])
        Q = 64 if "delta" in name else rng.choice([64, 128, 256])
        if "varlen" in name and "delta" not in name:
            P, N = 64, rng.choice([64, 128])
        H, b = int(2 ** rng.uniform(0, 20)), int(2 ** rng.uniform(0, 16))
        chunks = max(1, int(2 ** rng.uniform(18, 27) / (H * b)))
        T = rng.choice([1, chunks * Q, chunks * Q - Q // 2])
        G = rng.choice([g for g in (1, 2, max(1, H // 2), H) if H % g == 0])
        if "step" in name and rng.random() < 0.5:
            b, T = int(2 ** rng.uniform(0, 26)), 1
        call = scan_call(name, b, T, H, P, N, G, Q, rng.choice([ssd.SSD_BF16, ssd.SSD_F32]))
        if call is not None:
            calls.append(call)
    got = check(tmp_path, calls)
    assert 0 in got and UNSUPPORTED in got


def test_edges(tmp_path):
    """The most that is accepted, and one more."""
    bf, most = ssd.SSD_BF16, (1 << 24) - 1  # work-groups of 256 threads
    pairs = []
    for name in ("ssd_step", "ssd_diag_step", "ssd_delta_step"):
        pairs.append([scan_call(name, b, 1, 1, 16, 16, 1, 64, bf) for b in (most, most + 1)])
    for name in ("ssd_scan_fwd", "ssd_diag_scan_fwd", "ssd_scan_bwd", "ssd_diag_scan_bwd"):
        pairs.append([scan_call(name, 1, (H // 16) * 64, 16, 16, 16, 1, 64, bf) for H in (most - 15, most + 1)])  # chunks
        pairs.append([scan_call(name, 255, 1, H, 64, 256, 1, 64, bf) for H in (most // 16 // 255, most // 16 // 255 + 1)])  # states
    pairs.append([scan_call("ssd_scan_fwd_varlen", b, 1, 1024, 64, 64, 1, 64, bf) for b in (most // 1024, most // 1024 + 1)])
    for below, above in pairs:
        assert below is not None and above is not None
        assert check(tmp_path, [below, above]) == [0, UNSUPPORTED], (below[0], [(f, getattr(below[1], f)) for f, _ in below[1]._fields_])


def test_norm_and_pool(tmp_path):
    rng, calls = random.Random(7), []
    while len(calls) < 3000:
        P, N = rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128, 256])
        H, b = int(2 ** rng.uniform(0, 18)), int(2 ** rng.uniform(0, 24))
        T, G, dtype = int(2 ** rng.uniform(0, 9)), rng.choice([1, H]), rng.choice([ssd.SSD_BF16, ssd.SSD_F32])
        es = 2 if dtype == ssd.SSD_BF16 else 4
        if max(b * T * H * P, b * T * G * N, H * P * N) * es >= lr.FAR:
            continue
        at = [lr.FAKE + i * lr.FAR for i in range(14)]
        if rng.random() < 0.3:
            p = ssd.Norm(b, T, H, G, N, N // 4 if N >= 16 else 0, H * N, G * N, 1e-6, 0, 0, dtype)
            if b * T * H * N * es >= lr.FAR:
                continue
            calls.append(("ssd_bc_norm", p, at[:8] + [0]))
            ws = int(ssd._load().ssd_bc_norm_bwd_workspace_bytes(ctypes.byref(p)))
            calls.append(("ssd_bc_norm_bwd", p, at[:12] + [lr.FAKE + 30 * lr.FAR, ws, 0]))
            continue
        p = ssd.PoolProblem(b, T, H, P, N, G, H * P, G * N, G * N, 4, H * P * N, dtype, 0)
        kind = rng.choice(["step", "tree", "commit"])
        if kind == "step":  # x dt A B C D beta pool slots out y
            calls.append(("ssd_pool_step", p, at[:6] + [0] + at[7:11] + [0]))
        elif kind == "tree":  # x dt A B C D beta parents pool slots y
            calls.append(("ssd_tree_step", p, at[:5] + [0] + at[6:11] + [0]))
        else:  # x dt A B beta parents last pool slots out
            calls.append(("ssd_tree_commit", p, at[:10] + [0]))
    got = check(tmp_path, calls)
    assert 0 in got and UNSUPPORTED in got
