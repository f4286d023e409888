"""CPU tests of what the kernels' sources do not use, whatever the GPU they run on."""

import glob
import os

from paged_kv_decode_splitk_gb300 import build


def _sources():
    return {os.path.basename(p): open(p).read() for p in glob.glob(os.path.join(build.CSRC, "*"))}


def test_no_copy_or_signal_to_several_ctas():
    """Each CTA's copies and commits reach that CTA alone, so the same library serves replicas on several GPUs."""
    assert [name for name, text in _sources().items() if "multicast" in text] == []


def test_shared_prefix_pass_keeps_to_one_cta():
    """Its stages are given back by ordered arrivals at barriers of the same CTA."""
    for name, text in _sources().items():
        if name.startswith("pd_prefix"):
            for word in ("map_to_rank", "mbar_arrive_cluster", "relaxed"):
                assert word not in text, name
