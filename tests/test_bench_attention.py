"""CPU: how many launches the benchmark's attention variants count for a token (a trace summary takes that many
dispatches a token from the end)."""
import os

import pytest

import bench
from quant_dequant_gemv_amd import binding


def test_a_join_is_counted_only_where_there_is_one():
    heads = [("heads", ((), (None, None, 24, need))) for need in (0, 0, 1 << 20)]
    stream = [("plain", None), heads[0], ("swiglu", None), heads[1], heads[2], ("keep", [])]
    assert bench.attention_launches(stream) == 2 + 2 + 3


@pytest.mark.skipif(not os.path.exists(binding.LIB_PATH), reason="libqkgemv.so not built (run __graft_entry__.build())")
@pytest.mark.parametrize("context,split", [(1, False), (512, False), (32768, True), (262144, True)])
def test_short_contexts_are_not_cut(context, split):
    """The bench's layers: 24 heads on 4 of 256, pages of 64; up to 512 positions are one piece."""
    cache = binding.qk_kv_cache(1 << 28, 5000, 4, 256, 64)
    seqs = binding.qk_kv_seqs(1, 1, -(-context // 64), None, 1 << 20, 2 << 20)
    assert (binding.qk_kv_attn_workspace_bytes(cache, seqs, 24) > 0) == split
