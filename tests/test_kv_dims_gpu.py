"""Writing and reading at head dimensions that attention does not take: the library's own quantizers' codes and scales,
and its dequantized values.  (The sign of a zero is left out: the lanes' transform may give an exact zero the other one.)"""
import numpy as np
import pytest
import torch

import kv_ref
from test_kv_gpu import amax_of, fq, kv_rows, nv_with_scale  # noqa: F401  (fq: the fixture)

pytestmark = pytest.mark.gpu


def unsigned_zeros(codes):
    lo, hi = codes & 15, codes >> 4
    return torch.where(lo == 8, 0, lo) | torch.where(hi == 8, 0, hi) << 4


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,dim,page,rotate", [(1, 384, 7, True), (3, 640, 5, True), (2, 768, 16, True), (1, 896, 3, True),
                                                   (3, 160, 6, False)])
@pytest.mark.parametrize("base", [0, 512])
def test_other_head_dims(fq, fmt, dtype, heads, dim, page, rotate, base):  # noqa: F811
    """Planes at an allocation's start and 512 bytes on, where another would begin."""
    tokens, rng, block = 61, np.random.default_rng(dim), kv_ref.BLOCK[fmt]
    pages = 61 // page + 4
    k, v = (kv_rows(rng, tokens, heads, dim, dtype, "plain").cuda() for _ in range(2))
    (k_amax, kg), (v_amax, vg) = amax_of(2.0 ** -8), amax_of(0.00077)
    planes = []
    for width in (dim // 2, dim // block) * 2:
        store = torch.zeros(base + pages * heads * page * width, dtype=torch.uint8, device="cuda")
        planes.append(store[base:].view(pages, heads, page, width))
    cache = fq.KvCache(fmt, *planes, *(torch.tensor([g], dtype=torch.float32, device="cuda") for g in (kg, vg)))
    slots = torch.from_numpy(rng.permutation(pages * page)[:tokens].astype(np.int64)).cuda()
    rotation = "fwht128" if rotate else None
    print("write", fmt, dtype, heads, dim, page, rotate, base, flush=True)
    fq.kv_cache_write(cache, k, v, slots, rotation=rotation)
    for x, amax, c, s, rot in ((k, k_amax, planes[0], planes[1], rotate), (v, v_amax, planes[2], planes[3], False)):
        x = x.reshape(-1, dim)
        if rot:
            x = fq.fwht(x, transform_size=128)
        want = fq.quantize_mxfp4(x) if fmt == "mxfp4" else nv_with_scale(fq, x, amax)
        got = c.permute(0, 2, 1, 3).reshape(pages * page, -1)[slots].reshape(-1, dim // 2)
        assert torch.equal(unsigned_zeros(got), unsigned_zeros(want.codes))
        assert torch.equal(s.permute(0, 2, 1, 3).reshape(pages * page, -1)[slots].reshape(want.scales.shape), want.scales)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    n = pages * page
    got = fq.kv_cache_read(cache, table, torch.tensor([0, n], dtype=torch.int32, device="cuda"), total=n, rotation=rotation,
                           out_dtype=torch.float32)
    for x, g, c, s, rot in ((got[0], kg, planes[0], planes[1], rotate), (got[1], vg, planes[2], planes[3], False)):
        want = fq.dequantize(fmt, c.permute(0, 2, 1, 3).reshape(-1, dim // 2).contiguous(),
                             s.permute(0, 2, 1, 3).reshape(-1, dim // block).contiguous(),
                             torch.tensor([g], dtype=torch.float32, device="cuda") if fmt == "nvfp4" else None,
                             out_dtype=torch.float32)
        if rot:
            want = fq.fwht(want, transform_size=128)
        assert torch.equal(x.reshape(-1, dim), want)
