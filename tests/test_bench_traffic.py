"""The DRAM traffic that the bench reports beside a roofline is of the present kernels: an entry whose sources have changed is
taken again or taken out (it would be reported as null)."""
import pytest

import bench
from block_quantized_moe_router_gb300 import synth


@pytest.mark.parametrize("name", sorted(bench.TRAFFIC))
def test_no_stale_entry(name):
    cfg = synth.CONFIGS[name]
    kind = "decode" if cfg.T <= 8 else "tc" if cfg.act == synth.ACT_NVFP4 else "mma"
    assert bench.captured_traffic(name, bench.kernel_source_hash(bench.KERNEL_SOURCES[kind])) == bench.TRAFFIC[name][0]
