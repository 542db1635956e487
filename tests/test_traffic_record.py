"""The benchmark's step reports the measured HBM bytes of its products only while the
record was taken of the current kernel sources: it is, and parses."""

import bench


def test_the_traffic_record_is_of_the_current_sources():
    got = bench.measured_traffic("ffn_step_8192x4096x14336", 4)
    assert got is not None and 4.9e8 < got < 3e9           # no less than the operands and C
    assert bench.measured_traffic("ffn_step_8192x4096x14336", 5) is None
