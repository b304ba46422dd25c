"""The sources of the kernels whose CTAs work in pairs: what a warp writes to its CTA's shared memory for a product that the other CTA
issues is handed on at cluster scope. (Results cannot show it: an order that nothing promises may hold all the same.)"""
import os
import re

import pytest

from dsa_sparse_mla_gb300 import build


def source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["expanded.cu", "heads.cu"])
def test_writes_are_handed_on_at_cluster_scope(name):
    text = source(name)
    for fence in re.finditer(r"fence_proxy_async_smem\(\)", text):
        assert re.search(r"\b(\w*arrive\w*)\(", text[fence.end():]).group(1) == "arrive_writes"


def test_the_issuing_thread_waits_for_them():
    text = source("expanded.cu")
    for bar in ("v_full[ring.slot]", "p_full[b]", "unit_full[n % kPlaces]"):
        assert re.search(r"wait_writes\(&\w+(\.|->)%s," % re.escape(bar), text), bar


def test_what_the_forms_are():
    text = source("pair.cuh")
    release = text[text.index("void arrive_writes"):]
    assert release.index("fence_release_smem") < release.index("remote_arrive_relaxed")
    acquire = text[text.index("bool wait_cluster_smem"):]
    assert acquire.index("try_wait_relaxed") < acquire.index("fence_acquire_smem")
