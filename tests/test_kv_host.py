"""Host-side behaviour of the cache's entry points (no GPU compute)."""
import os

import pytest
import torch

from fp4_block_scaled_row_amd import _kv, _lib
from test_kv_abi import A, attention_args, cache, read_args, write_args


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libfp4q.so not built (run __graft_entry__.build())")
    return _lib.load()


def test_queries_without_a_sequence_are_refused(lib):
    """As a read of rows without a sequence is: they would be left as they are."""
    assert lib.fp4q_kv_attention(cache(), attention_args(seqs=0), A, 1 << 40, None) == _lib.FP4Q_ERR_INVALID_ARG
    assert lib.fp4q_kv_attention_workspace_bytes(cache(), attention_args(seqs=0)) == 0


@pytest.mark.parametrize("fmt", [_lib.FP4Q_NVFP4, _lib.FP4Q_MXFP4])
@pytest.mark.parametrize("head_dim", [384, 512, 640, 768, 896, 1024, 32, 64, 96, 160])
@pytest.mark.parametrize("base", [0x10000, 0x10200, 0x10400, 0x10600, 0x10800, 0x10A00, 0x10E00, 0x10001])
def test_scale_planes_of_dense_caches_lie_anywhere(lib, fmt, head_dim, base):
    """Writing and reading take scales a byte at a time: a dense cache is taken wherever its planes lie."""
    block = 16 if fmt == _lib.FP4Q_NVFP4 else 32
    row = head_dim // block
    c = cache(format=fmt, head_dim=head_dim, code_stride=(head_dim * 16, head_dim * 8, head_dim // 2),
              scale_stride=(row * 32, row * 16, row), k_scales=base, v_scales=base + 0x4000)
    assert lib.fp4q_kv_write(c, write_args(tokens=0), None) == _lib.FP4Q_OK
    assert lib.fp4q_kv_read(c, read_args(total=0), None) == _lib.FP4Q_OK


@pytest.mark.parametrize("fmt,head_dim,bytes_", [(_lib.FP4Q_NVFP4, 128, 2), (_lib.FP4Q_NVFP4, 256, 4),
                                                 (_lib.FP4Q_MXFP4, 128, 1), (_lib.FP4Q_MXFP4, 256, 2)])
def test_scale_planes_that_attention_loads_wide(lib, fmt, head_dim, bytes_):
    row = head_dim // (16 if fmt == _lib.FP4Q_NVFP4 else 32)
    for off in (0, 1, 2, 4):
        c = cache(format=fmt, head_dim=head_dim, code_stride=(head_dim * 16, head_dim * 8, head_dim // 2),
                  scale_stride=(row * 32, row * 16, row), k_scales=A + off)
        want = _lib.FP4Q_OK if off % bytes_ == 0 else _lib.FP4Q_ERR_UNSUPPORTED
        assert lib.fp4q_kv_attention(c, attention_args(total_q=0), None, 0, None) == want


class Handle:
    """What the Python entry points look at of a cache, on the CPU; calls to the library are recorded, not made."""
    head_dim, kv_heads, page_size, device, _index, _args = 128, 2, 16, torch.device("cpu"), -1, None


class Recorder:
    def __init__(self, calls):
        self.calls = calls

    def fp4q_kv_attention(self, cache, a, *rest):
        self.calls.append(a)
        return 0

    def fp4q_kv_attention_workspace_bytes(self, cache, a):
        self.calls.append(a)
        return 64


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(_kv._lib, "load", lambda: Recorder(made))
    monkeypatch.setattr(_kv, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(_kv, "_call", lambda cache, function, *args: function(*args))
    monkeypatch.setattr(_kv, "_workspaces", {(-1, 0): torch.zeros(64, dtype=torch.uint8)})
    return made


def attention(**kw):
    q, table = torch.zeros(6, 8, 128), torch.zeros(2, 4, dtype=torch.int32)
    cu = torch.tensor([0, 3, 6], dtype=torch.int32)
    return _kv.kv_cache_attention(q, Handle(), table, torch.zeros(2, dtype=torch.int32), cu_q=cu, **kw)


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1])
def test_numbers_past_32_bits_do_not_wrap(calls, value):
    """A window or a bound on the queries that is as good as none must not become a small one, or none at all."""
    attention(window=value, max_q=value)
    assert calls[-1].window == 2 ** 31 - 1 and calls[-1].max_q >= 6
    _kv.kv_cache_attention_workspace_bytes(torch.zeros(6, 8, 128), Handle(), torch.zeros(2, 4, dtype=torch.int32),
                                           max_q=value, window=value)
    assert calls[-1].window == 2 ** 31 - 1 and calls[-1].max_q >= 6


@pytest.mark.parametrize("value", [-1, -2 ** 31 - 1, -2 ** 32])
def test_negative_numbers_stay_negative(calls, value):
    attention(window=value, max_q=value)       # (for the library to refuse)
    assert calls[-1].window < 0 and calls[-1].max_q < 0


class Elsewhere(torch.Tensor):
    """A buffer that says it is on another GPU."""

    is_cuda = True

    def get_device(self):
        return 1


def test_a_workspace_of_another_device_is_refused(calls):
    with pytest.raises(ValueError, match="fp4q: the workspace"):
        attention(workspace=torch.zeros(1 << 20, dtype=torch.uint8).as_subclass(Elsewhere))
    with pytest.raises(ValueError, match="fp4q: the workspace"):
        attention(workspace=1 << 20)
    assert not calls
