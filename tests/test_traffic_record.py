"""The stored DRAM traffic of an assignment launch belongs to the kernel's current sources, without a
GPU: bench.py reports null where it does not, and the record has to be captured again."""

import os

from test_bench_host import ROOT, _bench


def test_stored_traffic_is_of_the_current_sources():
    b = _bench()
    record, found = b.load_traffic(b.kernel_source_sha())
    assert found is not None
    assert record is not None, "profiles/assign_kernel_traffic.txt is of other sources: capture it again"
    assert record["bytes_per_launch"] == record["dram_bytes_read"] + record["dram_bytes_write"]


def test_other_operators_are_none_of_the_kernel_s_sources():
    """What belongs to other kernels is declared elsewhere, so that its edits leave the record valid."""
    for rel in _bench().ASSIGN_KERNEL_SOURCES:
        with open(os.path.join(ROOT, rel)) as f:
            text = f.read()
        assert not any(word in text for word in ("launch_route", "launch_lookup", "launch_lists", "launch_clip"))
