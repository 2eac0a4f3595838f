"""The DRAM traffic that the bench reports is recorded per kernel and holds for the sources that it was
captured from: a change of those has to bring a new capture, or the bench reports none."""
import pytest

import bench


@pytest.mark.parametrize("call", sorted(bench.TRAFFIC_PROFILES))
def test_recorded_traffic_is_of_the_present_sources(call):
    bytes_per_launch = bench.recorded_traffic(call)
    assert bytes_per_launch is not None, f"{bench.TRAFFIC_PROFILES[call]} was captured from other GEMM sources"
    cost = bench.call_costs(8192, 2048, 768, 128, 8)[call]["bytes"]
    # every operand byte read once; of the results, those still in the L2 (129 MB) when the kernel ends are not counted
    assert cost - 129e6 <= bytes_per_launch <= 1.1 * cost
