"""Orders that the memory model asks of the kernels and no run can be relied on to show, read from their
sources: between two calls on a barrier, what has to stand there."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_attention_decode_indexer_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("start", ["auto issue_page = ", "auto issue_group = "])
def test_lanes_copies_are_tracked_before_the_stage_may_complete(start):
    """Lanes raise a stage's pending count with their asynchronous copies; lane 0 arrives for the stage
    behind a warp barrier (a warp reduction orders no memory)."""
    body = _source("decode_kernel.cuh").split(start)[1].split("return true;")[0]
    tracked, arrive = body.index("cp_async_mbar_arrive(&full[sb])"), body.index("mbar_arrive_expect_tx(&full[sb]")
    assert tracked < body.index("__syncwarp()") < arrive


def test_words_pushed_by_other_ctas_are_acquired_at_cluster_scope():
    """The heads' maxima of a whole page come from other CTAs by st.async, released at cluster scope."""
    store, common = _source("store_page_head.cu"), _source("common.cuh")
    assert "st.async.shared::cluster" in store
    assert re.findall(r"mbar_wait\S*\(&s_bar", store) == ["mbar_wait<true>(&s_bar"]
    cluster = common.split("if constexpr (CLUSTER)")[1].split("else")[0]
    assert "mbarrier.try_wait.parity.acquire.cluster.shared::cta" in cluster
