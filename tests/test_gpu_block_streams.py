"""The attention block's operators side by side: calls in flight on several streams, each with a workspace of its own,
two captured graphs that share one, calls back to back on one stream."""

import numpy as np
import pytest
import torch

from tests import test_gpu_kv_shared as shared, test_gpu_linear as linear
from tests.test_gpu_linear import m  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def linears(m, sizes, seed):  # noqa: F811
    """Calls of their own inputs and workspace, and what each gives alone."""
    out = []
    for i, (T, K, N, act) in enumerate(sizes):
        p = linear.problem(T, K, N, act=act, bias=True, seed=seed + i)
        a = [linear.on_gpu(p["x"]), torch.from_numpy(p["w"]).cuda(), torch.from_numpy(p["s"]).cuda()]
        b, ws = p["b"].cuda(), torch.zeros(m.linear_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")

        def call(a=a, b=b, ws=ws, act=act):
            return m.linear_a16w4_mxfp4(*a, bias=b, act=act, workspace=ws)

        want = call()
        linear.check(p, want)
        out.append((call, want, ws))
    return out


def test_streams_at_once(m):  # noqa: F811
    calls = linears(m, [(1, 512, 640, None), (400, 512, 2000, "silu"), (40, 2048, 300, None), (2000, 256, 1024, "swiglu")], 1)
    p = shared.problem(900, [40] * 30, [1] * 30, 2, 4, 64, 32, seed=3)
    alone = shared.run(m, p)
    shared.check(p, *alone)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    others = []
    for _ in range(15):
        for i, (call, _, _) in enumerate(calls):
            with torch.cuda.stream(streams[i]):
                got[i].append(call())
        others.append(shared.run(m, p))
    torch.cuda.synchronize()
    for (_, want, ws), outs in zip(calls, got):
        assert all(torch.equal(o, want) for o in outs)
        assert m.linear_read_status(ws) == 0
    for out, lse in others:
        assert torch.equal(out, alone[0]) and torch.equal(lse, alone[1])


@pytest.mark.parametrize("sizes", [((1500, 30), (300, 12)), ((1500, 60), (300, 50)), ((700, 90), (1500, 20))])
@pytest.mark.parametrize("tail", [0, 2000])  # (entries of the shared table past the prefix)
def test_two_graphs_share_a_workspace(m, sizes, tail):  # noqa: F811
    problems = [shared.problem(P, [20] * R, [1] * R, 2, 7, 128, 64, seed=R) for P, R in sizes]
    for p in problems:
        p["shared"] = np.concatenate([p["shared"], np.zeros(tail, np.int32)])
    ws, runs = None, []
    for p in problems:
        c = m.KvCacheMxfp4(p["pages"], 64, 2, 128, data=torch.from_numpy(p["data"]).cuda())
        q, R = p["q"].cuda(), len(p["lens"])
        args = [shared.i32(x) for x in (p["shared"], [p["P"]], p["table"], p["lens"], p["start"])]
        need = m.attention_shared_workspace_bytes(c, R, R, 14, p["table"].shape[1], 1, len(p["shared"]))
        if ws is None:
            ws = torch.zeros(need, dtype=torch.uint8, device="cuda")  # the larger of the two
        assert ws.numel() >= need
        out, lse = torch.empty_like(q), torch.empty(R, 14, device="cuda")

        def call(q=q, c=c, args=args, out=out, lse=lse):
            m.attention_kv_mxfp4_shared(q, c, *args, 1, scale=0.2, out=out, lse=lse, workspace=ws)

        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((g, p, out, lse, (q, c, args)))  # (the graph's inputs live as long as it does)
    for _ in range(5):
        for g, _, out, lse, _ in runs:
            out.zero_()
            g.replay()
        for _, p, out, lse, _ in runs:
            shared.check(p, out, lse)
    assert m.attention_read_status(ws) == 0


def test_back_to_back(m):  # noqa: F811
    """Chained on one stream without a wait between: each reads what the last wrote."""
    g = np.random.default_rng(5)
    x = torch.from_numpy(g.standard_normal((200, 512))).bfloat16().cuda()
    w = torch.from_numpy(g.integers(0, 256, (512, 256), dtype=np.uint8)).cuda()
    s = torch.from_numpy(g.integers(115, 119, (512, 16), dtype=np.uint8)).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def chain(sync):
        y = x
        for i in range(12):
            y = m.linear_a16w4_mxfp4(y[: (200, 20, 3)[i % 3]] if i % 4 == 3 else y, w, s, act="gelu", residual=None, workspace=ws)
            if sync:
                torch.cuda.synchronize()
        return y

    want = chain(True)
    for _ in range(10):
        assert torch.equal(chain(False), want)
