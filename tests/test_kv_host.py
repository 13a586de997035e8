"""Host-side behaviour of the cache's entry points (no GPU compute)."""
import os

import pytest

from fp4_block_scaled_row_amd import _lib
from test_kv_abi import A, attention_args, cache


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libfp4q.so not built (run __graft_entry__.build())")
    return _lib.load()


def test_queries_without_a_sequence_are_refused(lib):
    """As a read of rows without a sequence is: they would be left as they are."""
    assert lib.fp4q_kv_attention(cache(), attention_args(seqs=0), A, 1 << 40, None) == _lib.FP4Q_ERR_INVALID_ARG
    assert lib.fp4q_kv_attention_workspace_bytes(cache(), attention_args(seqs=0)) == 0
