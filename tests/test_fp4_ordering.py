"""The scopes of the CTA pairs' barriers, read in the sources: an order that is too weak
shows in no result, or in one of many runs, so it is looked for where it is written."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "routing_dispatch_expert_router_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_arrivals_at_the_other_ctas_barrier_have_cluster_scope():
    """Without a scope an arrival releases to its own CTA only."""
    arrive = re.findall(r'"mbarrier\.arrive[\w.:]*', source("ptx.cuh"))
    remote = [a for a in arrive if "shared::cluster" in a]
    assert len(remote) >= 3
    for a in remote:
        assert ".release.cluster." in a or ".relaxed.cluster." in a, a


@pytest.mark.parametrize("name,kernel,barriers", [
    ("grouped_gemm_fp4.cu", "grouped_gemm_fp4_pair_kernel(", "full empty scales tfull tempty"),
    ("grouped_gemm_fp4_bwd.cu", "fp4_dgrad_kernel(", "full empty tfull tempty")])
def test_waits_for_both_ctas_acquire_at_cluster_scope(name, kernel, barriers):
    """bar_*: the barriers that the other CTA, or MMAs that the other CTA issued, arrive at."""
    text = source(name)
    body = text[text.index(kernel):]
    body = body[:body.index("\n}\n")]
    for b in barriers.split():
        waits = re.findall(r"ptx::(mbar_wait\w*)\(bar_%s\b(?!_)" % b, body)
        assert waits and set(waits) == {"mbar_wait_cluster"}, (b, waits)


def test_values_made_for_the_other_ctas_mma_are_released():
    """The backward's converting warps write shared memory with plain stores: an arrival
    that orders tensor memory alone would not publish them."""
    body = source("grouped_gemm_fp4_bwd.cu")
    made = body[body.index("codes to values"):body.index("// ------------------------------------------------------------ epilogue")]
    assert "mbar_arrive_cluster_smem(leader_full" in made and "_cluster_tmem" not in made
    assert "fence_proxy_async_smem" in made
    ptx = source("ptx.cuh")
    f = ptx[ptx.index("void mbar_arrive_cluster_smem"):]
    f = f[:f.index("\n}\n")]
    assert f.index("fence.release.sync_restrict::shared::cta.cluster") < f.index("mbarrier.arrive")


def test_scale_columns_are_written_behind_a_tensor_memory_fence():
    """The columns' last readers are MMAs of the stage's turn before: between the barrier
    that says so and tcgen05.st stands the fence that orders them."""
    text = source("grouped_gemm_fp4.cu")
    f = text[text.index("void write_scales("):]
    f = f[:f.index("\n}\n")]
    assert "tc_fence_after" in f and f.index("tc_fence_after") < f.index("tmem_st")
    assert f.rindex("tmem_st_wait") < f.index("tc_fence_before")
