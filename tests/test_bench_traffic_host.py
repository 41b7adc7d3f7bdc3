"""The DRAM traffic that bench.py reports comes from captures of the current kernels' sources, so it is not left out."""
import bench
import workloads as W


def test_split_traffic_is_of_the_current_sources():
    assert bench.SPLIT_TRAFFIC_CAPTURED["source_hash"] == bench.kernel_source_hash()
    for name in bench.SPLIT_TRAFFIC_CAPTURED["configs"]:
        assert bench.ncu_traffic(name, W.CONFIGS[name]["tile_len"]) >= bench.config_algorithmic_bytes(name)


def test_prefill_traffic_is_of_the_current_sources():
    assert bench.PREFILL_TRAFFIC_CAPTURED["source_hash"] == bench.prefill_source_hash()
    assert bench.prefill_traffic() == bench.PREFILL_TRAFFIC_CAPTURED["read"] + bench.PREFILL_TRAFFIC_CAPTURED["write"]
