"""The bench line's DRAM traffic comes from a committed capture of the kernel sources in the tree."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_committed_traffic_is_of_the_present_sources():
    sys.path.insert(0, ROOT)
    import bench

    # a change of these sources needs a new capture (the command is in the file's note)
    for kernel, algorithmic in (("gate_up", 7.71e9), ("down", 4.49e9)):
        got = bench.measured_traffic("grok_prefill", kernel)
        assert got is not None, "profiles/dram_traffic.json was taken on other kernel sources"
        # at least the bytes that the kernel has to move, less what may stay in L2
        assert algorithmic - 126e6 <= got <= 3 * algorithmic
