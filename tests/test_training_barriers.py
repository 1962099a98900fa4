"""The training products' hand-over of tensor memory, read from the source: an
accumulator is overwritten only after both CTAs' reads of it.  The order is the
PTX ISA's for tcgen05 operations of different threads: wait::ld,
fence::before_thread_sync, an arrival; a wait, fence::after_thread_sync, the next
product; arrival and wait at cluster scope, for the arrivals come from the pair."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "video_vit_encoder_gb300", "csrc")


def _read(name):
    with open(os.path.join(SRC, name)) as f:
        return re.sub(r"//.*", "", f.read())


def _body(source, head):
    return re.search(head + r"\(.*?\n}", source, re.S).group()


def test_tensor_memory_is_handed_back_across_the_pair():
    s, common = _read("gemm_train.cuh"), _read("common.cuh")
    arrivals = re.findall(r"(\w+)\(tempty0 \+ 8 \* buf\)", s)
    assert arrivals == ["mbar_arrive_cluster_relaxed"]
    assert re.search(r"mbarrier\.arrive\.re\w+\.cluster\.shared::cluster", _body(s, "void mbar_arrive_cluster_relaxed"))
    waits = re.findall(r"(\w+)\(&tempty\[buf\]", s)
    assert waits == ["mbar_wait_cluster_relaxed"]
    assert re.search(r"mbarrier\.try_wait\.parity\.\w+\.cluster\.", _body(s, "bool mbar_wait_cluster_relaxed"))
    # the reads have completed and are fenced before any lane's arrival ...
    taken = re.search(r"auto chunk_taken = .*?};", s, re.S).group()
    assert re.search(r"tc_fence_before\(\);\s*__syncwarp\(\);\s*if \(lane == 0\) mbar_arrive", taken)
    assert "before_thread_sync" in _body(common, "void tc_fence_before")
    for loop in re.findall(r"load\(\w+, c, w(?:\[c\])?\);.*?chunk_taken", s, re.S):
        assert "tmem_wait_ld();" in loop
    for reader in ("void tmem_ld32f", "void slab_tile"):
        assert "tmem_wait_ld();" in _body(s, reader)
    # ... and the next product comes after the wait and its fence
    after = s[s.index("mbar_wait_cluster_relaxed(&tempty[buf]"):]
    assert after.index("tc_fence_after();") < after.index("umma_f16_ss_pair_warp(")
    assert "after_thread_sync" in _body(common, "void tc_fence_after")
