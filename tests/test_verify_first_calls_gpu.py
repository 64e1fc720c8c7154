"""The first calls of a process, made by several threads at the same time: each asks what its kernels' launches rest on, and takes
the same launch as any later call."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import threading, torch
import paged_kv_cache_83_gb300 as pa
from tests.test_verify_gpu import Drafts
pa.load()
cases = [Drafts([1 + s % 3, 2, 4], 30000 + 1000 * s, ("f32", "bf16")[s % 2], certain=s % 4 > 1, seed=s) for s in range(8)]
streams = [torch.cuda.Stream() for _ in cases]
torch.cuda.synchronize()
together, failed = threading.Barrier(len(cases)), []
def call(d, s):
    try:
        together.wait()
        d.run(stream=s)
    except Exception as e:
        failed.append(e)
threads = [threading.Thread(target=call, args=a) for a in zip(cases, streams)]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
assert not failed, failed
for d in cases:
    acc, nxt = d.wanted()
    assert d.accepted.tolist() == acc and d.next.tolist() == nxt and int(d.err) == 0
    d.check()
print("equal")
"""


def test_several_threads_at_once():
    for _ in range(2):
        r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=Path(__file__).resolve().parents[1], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-2000:]
