"""The give-up path of the attention kernels' bounded waits, run on the GPU without a fault.

The wait hook (moe_set_wait_limit) gives the next call a 1 ms limit and makes its waits for cache records (streaming
kernel) and for a tile's weights (tensor-core kernel) expect one arrival more than will come, so the real wait code runs
out: the kernels must record MOE_STATUS_WAIT_TIMEOUT, stop and return, and the next calls on the workspace are right.
"""

import ctypes
import os
import re
import time

import pytest
import torch

from tests.conftest import ROOT
from tests.test_gpu_kv_attention import check, i32, m, problem  # noqa: F401  (m: the fixture)

CASES = {
    "streamed, few requests": dict(lens=[300, 5, 2000], qlens=[1, 1, 1], H=2, G=4, D=128, page=64),
    "streamed, many requests": dict(lens=[90] * 50, qlens=[1] * 50, H=2, G=2, D=64, page=16),
    "prompts": dict(lens=[300, 128, 520, 90], qlens=[60, 128, 300, 1], H=40, G=1, D=128, page=64),
    "prompts, heads of 64": dict(lens=[700, 40, 300, 90], qlens=[300, 40, 257, 40], H=40, G=1, D=64, page=32),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_waits_that_run_out_end_the_call(m, name):  # noqa: F811
    p = problem(**CASES[name])
    c = m.KvCacheMxfp4(p["pages"], p["page"], p["H"], p["D"], data=torch.from_numpy(p["data"]).cuda())
    q, args = p["q"].cuda(), (i32(p["table"]), i32(p["lens"]), i32(p["start"]))
    most = int((p["start"][1:] - p["start"][:-1]).max())
    ws = torch.zeros(m.attention_workspace_bytes(c, len(p["lens"]), q.shape[0], q.shape[1], p["table"].shape[1], most),
                     dtype=torch.uint8, device="cuda")

    def call():
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        m.attention_kv_mxfp4(q, c, *args, most, scale=0.01, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        return out, lse

    check(p, *call(), 0.01)
    assert m.attention_read_status(ws) == 0
    lib = m._native.load()
    for _ in range(2):
        assert lib.moe_set_wait_limit(ctypes.c_uint64(1_000_000), 1) == 0
        t0 = time.perf_counter()
        call()  # the outputs are invalid
        assert time.perf_counter() - t0 < 1.5  # the 1 ms limit, not the 2 s default, ended the waits
        assert m.attention_read_status(ws) == m.MOE_STATUS_WAIT_TIMEOUT
        # the hook is gone, the workspace serves the next calls
        for _ in range(2):
            check(p, *call(), 0.01)
        assert m.attention_read_status(ws) == 0


@pytest.mark.parametrize("name", ["kv_stream.cu", "kv_prompt.cu"])
def test_every_wait_gives_one_result_a_warp(name):
    """mbar_wait's result differs between lanes that run out of time one by one; a branch on it would leave lanes behind
    in the next collective.  Read off the sources: waits are the warp's (mbar_wait_warp) or voted on."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(ROOT, "mxfp4_weight_only_gb300", "csrc", name)).read())
    text = text.replace("mbar_wait_warp", "")
    for s in re.split(r"[;{}]", text):
        if "mbar_wait(" not in s and "mbar_try_wait" not in s:
            continue
        if re.search(r"\b(all\(|__all_sync\(0xffffffffu, )mbar_", s):
            continue
        # kept, not branched on, until a vote ends the loop's body
        assert re.match(r"\s*ok = ", s), s
        rest = text[text.index(s) + len(s):]
        rest = rest[:re.search(r"ok = __all_sync\(0xffffffffu, ok\) != 0;\s*}", rest).start()]
        assert not re.search(r"\bbreak;|\bif \(!ok\)|return", rest), s
