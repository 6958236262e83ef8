"""The attention block's operators called by several host threads at once, the first calls of the process among them: each
with a stream and workspace of its own, in a child process, so that nothing has been loaded or asked for before."""

import os
import subprocess
import sys

import pytest

from tests.conftest import ROOT
from tests.test_gpu_linear import m  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

CHILD = """
import threading
import torch
import mxfp4_weight_only_gb300 as m

torch.cuda.init()
g = torch.Generator(device="cuda").manual_seed(1)
u8 = dict(device="cuda", dtype=torch.uint8, generator=g)


def linear(T, K, N):
    x = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    w, s = torch.randint(0, 256, (N, K // 2), **u8), torch.randint(115, 122, (N, K // 32), **u8)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return lambda stream: m.linear_a16w4_mxfp4(x, w, s, act="silu", workspace=ws, stream=stream)


def shared(R, tokens):
    c = m.KvCacheMxfp4(40 + R, 16, 2, 64)
    c.data.random_(0, 120)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    q = torch.randn(R, 16, 64, device="cuda", generator=g).bfloat16()
    args = (q, c, i32(list(range(40)) + [-1] * (tokens // 16)), i32([640]), i32([[40 + r] for r in range(R)]), i32([9] * R),
            i32(list(range(R + 1))), 1)
    ws = torch.zeros(m.attention_shared_workspace_bytes(c, R, R, 16, 1, 1, len(args[2])), dtype=torch.uint8, device="cuda")
    return lambda stream: m.attention_kv_mxfp4_shared(*args, scale=0.05, workspace=ws, stream=stream)


calls = [linear(600, 256, 4000), linear(40, 2912, 2500), linear(300, 4128, 600), linear(24, 512, 700), linear(3, 256, 9000),
         shared(3, 0), shared(60, 131072), shared(60, 131072)]
torch.cuda.synchronize()
gate, results, errors = threading.Barrier(len(calls)), [None] * len(calls), []


def work(i):
    try:
        stream = torch.cuda.Stream()
        gate.wait()
        out = [calls[i](stream) for _ in range(30)]
        stream.synchronize()
        results[i] = out
    except Exception as e:
        errors.append(repr(e))
        gate.abort()


threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert not errors, errors
for call, outs in zip(calls, results):
    want = call(None)
    assert all(torch.equal(o, want) for o in outs) and torch.isfinite(want.float()).all()
print("agree")
"""


def test_first_calls_at_once(m):  # noqa: F811
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": ROOT})
    assert r.returncode == 0 and r.stdout.strip().endswith("agree"), r.stdout + r.stderr
