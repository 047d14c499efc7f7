"""The DRAM traffic that the bench reports is of the GEMM sources in the tree."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


def test_capture_is_of_the_current_sources():
    import bench
    with open(bench.PROFILE_TRAFFIC) as f:
        entries = {k: v for k, v in json.load(f).items() if not k.startswith("_")}
    assert "g1_up_swiglu@mixtral" in entries
    assert {k for k, v in entries.items() if v["source_hash"] != bench.source_hash()} == set()


def test_attention_code_is_not_in_the_hashed_sources():
    """So that work on the attention operators leaves the capture valid."""
    for f in ("api.cu", "common.cuh"):
        with open(os.path.join(ROOT, "token_dispatch_grouped_gb300", "csrc", f)) as fh:
            src = fh.read()
        assert "namespace attn" not in src and "attn" not in src and "moe_attention.h" not in src
