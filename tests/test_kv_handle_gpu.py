"""Cache handles made by kv_cache()."""
import pytest
import torch

from test_kv_gpu import fq  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("default", [torch.float32, torch.bfloat16, torch.float64])
def test_tensor_scales_whatever_the_default_dtype_is(fq, default):  # noqa: F811
    """A model made under torch.set_default_dtype makes its cache there too."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        cache = fq.kv_cache(2, 16, 1, 64, k_global=0.25, v_global=2.0 ** -9)
    finally:
        torch.set_default_dtype(before)
    assert cache.k_global.dtype == cache.v_global.dtype == torch.float32
    assert cache.k_global.item() == 0.25 and cache.v_global.item() == 2.0 ** -9
