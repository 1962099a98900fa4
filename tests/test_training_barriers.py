"""The training products' hand-over of tensor memory, read from the source: an
accumulator is overwritten only after both CTAs' reads of it, which their
arrivals release and the issuing warp's wait acquires, at cluster scope."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "video_vit_encoder_gb300", "csrc")


def _read(name):
    with open(os.path.join(SRC, name)) as f:
        return f.read()


def test_tensor_memory_is_released_and_acquired_across_the_pair():
    s = _read("gemm_train.cuh")
    assert "relaxed" not in re.sub(r"//.*", "", s)
    arrivals = re.findall(r"(\w+)\(tempty0 \+ 8 \* buf\)", s)
    assert arrivals == ["mbar_arrive_cluster"]
    assert "mbarrier.arrive.release.cluster" in re.search(r"void mbar_arrive_cluster\(.*?\n}", _read("common.cuh"), re.S).group()
    waits = re.findall(r"(\w+)\(&tempty\[buf\]", s)
    assert waits == ["mbar_wait_cluster"]
    assert "mbarrier.try_wait.parity.acquire.cluster" in re.search(r"bool mbar_wait_cluster\(.*?\n}", s, re.S).group()
