"""The ncu record that bench.py reports as `roofline.traffic` belongs to the attention kernel's present source."""
import bench
from query_union_paged_b200 import workloads as W


def test_recorded_traffic_is_of_the_present_kernel_source():
    for config in ("2", "3", "4a", "4b", "4c", "5", "6"):
        name = {"2": "gqa_chunk_bf16_16k+2k", "3": "gqa_chunk_fp8_16k+2k", "4a": "ctx64k_fp8_mixa",
                "4b": "ctx64k_fp8_mixb", "4c": "ctx64k_fp8_mixc", "5": "block_union_bf16_128k+1k",
                "6": "chunk16k_fp8_16k+16k"}[config]
        assert config in W.CONFIGS and bench.profiled_traffic(name) > 4e7, name
