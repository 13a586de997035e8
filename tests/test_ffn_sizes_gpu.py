"""Calls of more workgroups than one dimension of a launch takes."""
import numpy as np
import pytest
import torch

import ffn_ref
from test_ffn_gpu import check, fq, sum_bound, values  # noqa: F401

pytestmark = pytest.mark.gpu


def test_norm_of_more_rows_than_a_dimension_has_waves(fq):
    """2^26 rows and some (a wave each): every row, against fp32 of torch."""
    print("norm of many short rows", flush=True)
    rows, d = (1 << 26) + 3, 8
    x = torch.randn(rows, d, device="cuda").bfloat16()
    w = torch.randn(d, device="cuda").bfloat16()
    y = fq.rms_norm(x, w).out
    for at in range(0, rows, 1 << 24):
        v = x[at:at + (1 << 24)].float()
        want = v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.float()
        # half a step of bf16, and fp32's few roundings on either side
        assert bool(((y[at:at + (1 << 24)].float() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs()).all())


def test_norm_of_more_rows_than_a_dimension_has_workgroups(fq):
    """Rows with a workgroup each, quantized, the same one again and again but for the first and last of every 2^21."""
    print("norm of many rows, a workgroup each", flush=True)
    rows, d = (1 << 24) + 5, 1056
    one = torch.randn(1, d, device="cuda").bfloat16()
    w = torch.ones(d, device="cuda")
    n = fq.rms_norm(one.expand(rows, d), w, quantize="mxfp8").out
    want = fq.rms_norm(one, w, quantize="mxfp8").out
    for got, first in zip(n, want):
        for part in got.split(1 << 20):
            assert bool((part == first).all())


def test_one_row_of_more_outputs_than_a_dimension_has_threads(fq):
    """A token's products with 2^28 and some rows of the weight: 32 rows and 512 threads a workgroup."""
    print("one row, many outputs", flush=True)
    n, k = (1 << 28) + 37, 32
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    codes = torch.randint(0, 256, (n, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.full((n, 1), 127, device="cuda", dtype=torch.uint8)
    x = torch.randn(1, k, device="cuda")
    y = fq.fp4_linear(x, fq.Fp4Weight("mxfp4", codes, scales))
    torch.cuda.synchronize()
    # ones of the first, last and some rows between, and those around every border of 2^21 workgroups of 16 and 32
    at = np.unique(np.concatenate([np.r_[0:64, n - 64:n], np.random.default_rng(0).integers(0, n, 4096)] + [
        np.arange(b - 40, b + 40) for b in range(1 << 25, n, 1 << 25)]))
    at = at[at < n]
    pick = torch.from_numpy(at).cuda()
    v = values("mxfp4", (codes[pick].cpu().numpy(), scales[pick].cpu().numpy(), None))
    xv = x.double().cpu().numpy()
    want, S = (xv @ v.T)[0], (np.abs(xv) @ np.abs(v).T)[0]
    check(y[0][pick], want, sum_bound(S, k, 3) + 2.0 ** -24 * np.abs(want))


def test_gated_weight_whose_scales_pass_2_31_bytes(fq):
    """65 rows over two factors of 8388607, NVFP4: the second one's scales begin 256 bytes below 2^31."""
    print("gated, scales past 2^31", flush=True)
    rows, half, k = 65, 8388607, 4096
    n = 2 * half
    if torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved() - torch.cuda.memory_allocated() < 60 << 30:
        pytest.skip("60 GiB of GPU memory")
    assert half * (k // 16) < 1 << 31 < (half + 127) * (k // 16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    # (rows repeat: each is one of 2^16, in an order that puts no two tiles' rows alike)
    some = torch.randint(0, 256, (1 << 16, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    low = torch.randint(0x18, 0x49, (1 << 16, k // 16), generator=gen, device="cuda", dtype=torch.uint8)
    codes = torch.empty(n, k // 2, device="cuda", dtype=torch.uint8)
    scales = torch.empty(n, k // 16, device="cuda", dtype=torch.uint8)
    for at in range(0, n, 1 << 16):
        size, turn = min(1 << 16, n - at), 37 * (at >> 16)
        codes[at:at + size] = some.roll(turn, 0)[:size]
        scales[at:at + size] = low.roll(-turn, 0)[:size]
    x = torch.randn(rows, k, generator=gen, device="cuda").bfloat16()
    g = torch.full((1,), 0.01 / k ** 0.5, device="cuda")
    h = fq.fp4_gated(x, fq.Fp4Weight("nvfp4", codes, scales, g))
    torch.cuda.synchronize()
    at = np.unique(np.r_[0:200, half - 200:half, np.random.default_rng(0).integers(0, half, 1500)])
    assert 0 <= at.min() and at.max() < half
    pick = torch.from_numpy(at).cuda()
    xv = x.double().cpu().numpy()
    both = [values("nvfp4", (codes[i].cpu().numpy(), scales[i].cpu().numpy(), g.item())) for i in (pick, pick + half)]
    (p, u), (tp, tu) = ([f(xv, v) for v in both] for f in (
        lambda a, v: a @ v.T, lambda a, v: sum_bound(np.abs(a) @ np.abs(v).T, k, 1)))
    want = ffn_ref.gated(p, u)
    # SiLU's slope is at most 1.1
    check(h[:, pick], want, 1.1 * tp * (np.abs(u) + tu) + (np.abs(p) + tp) * tu + (2.0 ** -8 + 2.0 ** -21) * np.abs(want))
