"""Host-side checks of the cache's C ABI (no GPU compute): bad arguments are
refused with the documented status before anything is enqueued.  The addresses
are made up and never followed."""
import ctypes as C
import math
import os

import pytest

from fp4_block_scaled_row_amd import _lib

A = 0x10000         # an aligned address


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libfp4q.so not built (run __graft_entry__.build())")
    return _lib.load()


def fields(obj, **kw):
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(obj, k)[:] = v
        else:
            setattr(obj, k, v)
    return obj


def cache(**kw):
    c = _lib.KvCacheArgs()
    fields(c, format=_lib.FP4Q_NVFP4, kv_heads=2, head_dim=128, page_size=16, num_pages=8, k_codes=A, k_scales=A,
           v_codes=A, v_scales=A, k_global=A, v_global=A, code_stride=(2048, 1024, 64), scale_stride=(256, 128, 8))
    return fields(c, **kw)


def write_args(**kw):
    a = _lib.KvWriteArgs()
    fields(a, tokens=4, k=A, v=A, k_stride=(256, 128), v_stride=(256, 128), slots=A, in_dtype=_lib.FP4Q_BF16,
           rotation=_lib.FP4Q_ROT_NONE)
    return fields(a, **kw)


def read_args(**kw):
    a = _lib.KvReadArgs()
    fields(a, page_table=A, table_stride=4, table_cols=4, seqs=2, cu=A, total=10, k_out=A, v_out=A,
           out_dtype=_lib.FP4Q_BF16, rotation=_lib.FP4Q_ROT_NONE)
    return fields(a, **kw)


def attention_args(**kw):
    a = _lib.KvAttentionArgs()
    fields(a, q=A, q_stride=(1024, 128), out=A, cu_q=A, seq_lens=A, page_table=A, table_stride=4, total_q=6,
           table_cols=4, seqs=2, max_q=3, q_heads=8, dtype=_lib.FP4Q_BF16, causal=1, window=0,
           rotation=_lib.FP4Q_ROT_NONE, scale=0.1)
    return fields(a, **kw)


INVALID, UNSUPPORTED = "FP4Q_ERR_INVALID_ARG", "FP4Q_ERR_UNSUPPORTED"
BAD_CACHES = [
    (dict(format=7), INVALID), (dict(format=-1), INVALID), (dict(format=_lib.FP4Q_IF4), UNSUPPORTED),
    (dict(kv_heads=0), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=100), INVALID),
    (dict(head_dim=2048), UNSUPPORTED), (dict(page_size=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(num_pages=-3), INVALID), (dict(num_pages=1 << 31), UNSUPPORTED), (dict(kv_heads=5000), UNSUPPORTED),
    (dict(k_codes=None), INVALID), (dict(v_scales=None), INVALID), (dict(k_global=None), INVALID),
    (dict(v_global=None), INVALID), (dict(k_codes=A + 8), UNSUPPORTED), (dict(v_scales=A + 1), UNSUPPORTED),
    (dict(code_stride=(2048, 1024, 72)), UNSUPPORTED), (dict(code_stride=(-2048, 1024, 64)), INVALID),
    (dict(code_stride=(1 << 31, 1024, 64)), UNSUPPORTED), (dict(scale_stride=(256, 128, 9)), UNSUPPORTED),
    (dict(scale_stride=(256, -128, 8)), INVALID),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES, ids=str)
def test_caches(lib, kw, status):
    want = getattr(_lib, status)
    for call, args in ((lib.fp4q_kv_write, write_args()), (lib.fp4q_kv_read, read_args())):
        assert call(cache(**kw), args, None) == want
    assert lib.fp4q_kv_attention(cache(**kw), attention_args(), A, 1 << 40, None) == want
    assert lib.fp4q_kv_attention_workspace_bytes(cache(**kw), attention_args()) == 0


def test_no_structures(lib):
    for call, args in ((lib.fp4q_kv_write, write_args()), (lib.fp4q_kv_read, read_args())):
        assert call(None, args, None) == _lib.FP4Q_ERR_INVALID_ARG
        assert call(cache(), None, None) == _lib.FP4Q_ERR_INVALID_ARG
    assert lib.fp4q_kv_attention(None, attention_args(), A, 1 << 40, None) == _lib.FP4Q_ERR_INVALID_ARG
    assert lib.fp4q_kv_attention(cache(), None, A, 1 << 40, None) == _lib.FP4Q_ERR_INVALID_ARG
    assert lib.fp4q_kv_attention_workspace_bytes(None, None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), INVALID), (dict(in_dtype=9), INVALID), (dict(rotation=17), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(k_stride=(-256, 128)), INVALID),
    (dict(v_stride=(256, 132)), UNSUPPORTED), (dict(k=A + 2), UNSUPPORTED), (dict(slots=A + 4), UNSUPPORTED),
], ids=str)
def test_write(lib, kw, status):
    assert lib.fp4q_kv_write(cache(), write_args(**kw), None) == getattr(_lib, status)


def test_rotation_needs_whole_chunks(lib):
    c = cache(head_dim=96, code_stride=(1536, 768, 48), scale_stride=(192, 96, 6))
    r = _lib.FP4Q_ROT_FWHT128
    assert lib.fp4q_kv_write(c, write_args(rotation=r), None) == _lib.FP4Q_ERR_UNSUPPORTED
    assert lib.fp4q_kv_read(c, read_args(rotation=r), None) == _lib.FP4Q_ERR_UNSUPPORTED
    assert lib.fp4q_kv_attention(c, attention_args(rotation=r), A, 1 << 40, None) == _lib.FP4Q_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(total=-1), INVALID), (dict(seqs=-1), INVALID), (dict(seqs=0), INVALID), (dict(table_cols=-1), INVALID),
    (dict(table_stride=3), INVALID), (dict(out_dtype=9), INVALID), (dict(rotation=-1), INVALID), (dict(cu=None), INVALID),
    (dict(page_table=None), INVALID), (dict(k_out=A + 4), UNSUPPORTED), (dict(v_out=A + 8), UNSUPPORTED),
], ids=str)
def test_read(lib, kw, status):
    assert lib.fp4q_kv_read(cache(), read_args(**kw), None) == getattr(_lib, status)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=9), INVALID), (dict(total_q=-1), INVALID), (dict(seqs=-1), INVALID), (dict(q_heads=0), INVALID),
    (dict(q_heads=7), INVALID), (dict(table_cols=-1), INVALID), (dict(table_stride=3), INVALID), (dict(window=-1), INVALID),
    (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID), (dict(window=4, causal=0), UNSUPPORTED),
    (dict(rotation=99), INVALID), (dict(max_q=-1), INVALID), (dict(cu_q=None), INVALID), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(seq_lens=None), INVALID), (dict(page_table=None), INVALID),
    (dict(q_stride=(-1024, 128)), INVALID), (dict(q_stride=(1024, 132)), UNSUPPORTED), (dict(q=A + 2), UNSUPPORTED),
    (dict(out=A + 8), UNSUPPORTED), (dict(seqs=70000), UNSUPPORTED), (dict(total_q=1 << 29), UNSUPPORTED),
    # (more pieces of work than 31 bits count)
    (dict(seqs=60000, total_q=1 << 27, max_q=2000, table_cols=1 << 20, table_stride=1 << 20), UNSUPPORTED),
], ids=str)
def test_attention(lib, kw, status):
    a = attention_args(**kw)
    assert lib.fp4q_kv_attention(cache(), a, A, 1 << 40, None) == getattr(_lib, status)
    assert lib.fp4q_kv_attention_workspace_bytes(cache(), a) == 0


@pytest.mark.parametrize("head_dim", [32, 160, 512, 1024])
def test_attention_head_dims(lib, head_dim):
    c = cache(head_dim=head_dim, code_stride=(1 << 16, 1 << 15, 1024), scale_stride=(1 << 14, 1 << 13, 512))
    assert lib.fp4q_kv_attention(c, attention_args(), A, 1 << 40, None) == _lib.FP4Q_ERR_UNSUPPORTED


def test_nothing_to_do(lib):
    assert lib.fp4q_kv_write(cache(), write_args(tokens=0, k=None, v=None, slots=None), None) == _lib.FP4Q_OK
    assert lib.fp4q_kv_read(cache(), read_args(total=0), None) == _lib.FP4Q_OK
    assert lib.fp4q_kv_read(cache(), read_args(k_out=None, v_out=None), None) == _lib.FP4Q_OK
    assert lib.fp4q_kv_attention(cache(), attention_args(total_q=0), None, 0, None) == _lib.FP4Q_OK
    assert lib.fp4q_kv_attention(cache(), attention_args(seqs=0, total_q=0), None, 0, None) == _lib.FP4Q_OK
