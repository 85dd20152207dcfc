"""The package offers the operators of a speculative decoding step as it does the library's others."""
import pytest

import paged_kv_cache_95_gb300 as package
from paged_kv_cache_95_gb300 import pagedkv

STEP = ["rotary_frequencies", "rotary_embedding", "rotary_reshape_and_cache", "rotary_reshape_and_cache_fp8",
        "paged_attention_tree", "paged_attention_tree_workspace_size", "speculative_verify", "kv_compact_path"]


@pytest.mark.parametrize("name", STEP)
def test_step_operators(name):
    assert getattr(package, name) is getattr(pagedkv, name)


def test_step_limits():
    assert package.MAX_TREE_NODES == 64
