"""The launches that an entry point would make, on the host (tests/launches/record.c)."""
import os
import subprocess

import ssd_chunked_scan_03_amd as ssd

HERE = os.path.dirname(os.path.abspath(__file__))
MOST = 0xffffffff  # threads of one launch along one dimension of its grid
FAKE = 1 << 50     # operands lie FAKE + k FAR apart; nothing reads them
FAR = 1 << 42


def recorder(folder):
    exe = os.path.join(str(folder), "record")
    subprocess.run(["gcc", "-O1", "-std=gnu11", "-rdynamic", os.path.join(HERE, "launches", "record.c"), "-ldl", "-o", exe],
                   check=True, capture_output=True, text=True)
    return exe


def record(exe, calls, show=0):
    """calls: (entry point, descriptor, the other arguments) -> for each (status, [(grid, work-group, first argument's bytes)])."""
    lines = [" ".join([name, bytes(p).hex(), str(show), *(str(v) for v in args)]) for name, p, args in calls]
    r = subprocess.run([exe, ssd.library_path()], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    out, launches = [], []
    for line in r.stdout.splitlines():
        v = line.split()
        if v[0] == "launch":
            launches.append((tuple(map(int, v[1:4])), tuple(map(int, v[4:7])), bytes.fromhex(v[7]) if len(v) > 7 else b""))
        else:
            out.append((int(v[1]), launches))
            launches = []
    assert len(out) == len(calls)
    return out


def fits(launches):
    return all(g * w <= MOST for grid, group, _ in launches for g, w in zip(grid, group))
