"""Barriers of the attention kernels, read off their sources: between the thread that initialises mbarriers and the
first use by another thread stands a barrier that orders memory (a shuffle or a vote does not)."""

import os
import re

import pytest

from tests.conftest import ROOT


def code(name):
    text = open(os.path.join(ROOT, "mxfp4_weight_only_gb300", "csrc", name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name,until", [
    ("kv_stream.cu", "grid_dep_launch_dependents();"),  # nothing after it syncs on the way of up to 32 requests
    ("kv_prompt.cu", "prompt_item<D, true>"),
])
def test_initialised_barriers_are_published(name, until):
    text = code(name)
    body = text[text.index("fence_barrier_init();"):]
    body = body[:body.index(until)]
    assert re.search(r"__sync(warp|threads)\(\);", body), name
