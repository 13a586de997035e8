"""The bounds of the linear layers' 32-bit arithmetic (csrc/fp4q_ffn_sizes.h), compiled by themselves and held against
the arithmetic of the kernels that rely on them, written again here."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

import fp4_block_scaled_row_amd  # noqa: F401
from fp4_block_scaled_row_amd import _lib, build
from test_ffn_abi import OK, UNSUPPORTED, lib, linear_args, weight  # noqa: F401

SOURCE = r"""
#include "fp4q_ffn_sizes.h"
extern "C" int scales_fit(int gated, int64_t n, int64_t k) { return fp4q::ring_scales_fit(gated, n, k); }
extern "C" unsigned grid_x(int64_t groups) { return fp4q::grid_x(groups); }
extern "C" unsigned grid_y(int64_t groups) { return fp4q::grid_y(groups); }
extern "C" int tiles_fit(int64_t tiles) { return fp4q::tiles_fit(tiles); }
extern "C" int few_eight_fits(int64_t rows, int64_t k) { return fp4q::few_eight_fits(rows, k); }
extern "C" int64_t grid_row() { return fp4q::kGridRow; }
"""


@pytest.fixture(scope="module")
def sizes(tmp_path_factory):
    at = tmp_path_factory.mktemp("sizes")
    (at / "sizes.cpp").write_text(SOURCE)
    cxx = shutil.which("g++") or build.hipcc()
    r = subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I" + build.CSRC, str(at / "sizes.cpp"), "-o",
                        str(at / "sizes.so")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = C.CDLL(str(at / "sizes.so"))
    lib.scales_fit.argtypes = [C.c_int, C.c_int64, C.c_int64]
    for f in (lib.grid_x, lib.grid_y, lib.tiles_fit):
        f.argtypes = [C.c_int64]
    lib.few_eight_fits.argtypes = [C.c_int64, C.c_int64]
    lib.grid_x.restype = lib.grid_y.restype = C.c_uint
    lib.grid_row.restype = C.c_int64
    return lib


def largest_scale_offset(n, k, block):
    """The last byte that a thread of the gated ring kernel asks for, from the tile's first scale of the first factor:
    local row 255 of the tile is row 127 of its factor, and a thread has 4 bytes at most."""
    half, srow = n // 2, k // block
    w_row = min(127, half - 1)
    return (half + w_row) * srow + srow - 1


@pytest.mark.parametrize("k", [64, 128, 4096, 16384, 1 << 20, 1 << 22])
def test_gated_scale_offsets_stay_in_32_bits(sizes, k):
    """At and around the largest weight that is taken; sizes well inside it are."""
    edge = (1 << 31) // (k // 16)                  # half the rows at which the second factor's first scale is past 2^31
    for half in {edge + d for d in range(-300, 300)} | {edge // 2, 1, 127, 128}:
        if half < 1 or 2 * half >= 1 << 31:
            continue
        if sizes.scales_fit(1, 2 * half, k):
            for block in (16, 32):
                assert largest_scale_offset(2 * half, k, block) < 1 << 31, (half, k, block)
        if half <= edge - 129:
            assert sizes.scales_fit(1, 2 * half, k)


@pytest.mark.parametrize("n,k", [(16777214, 4096), (2 * 2097151, 16384)])
def test_gated_weights_just_below_2_31_scales_go_another_way(sizes, n, k):
    """Second factors that begin below 2^31 and end past it."""
    assert n // 2 * (k // 16) < 1 << 31 <= largest_scale_offset(n, k, 16)
    assert not sizes.scales_fit(1, n, k)


def test_other_directions_have_no_second_factor(sizes):
    assert sizes.scales_fit(0, (1 << 31) - 1, 1 << 22)


# ---- grids: a dimension has fewer than 2^32 threads (workgroups of 1024 at most) and 65535 workgroups in y

@pytest.mark.parametrize("groups", [1, 255, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, (1 << 22) + 5, 1 << 24, 1 << 26,
                                    (1 << 31) - 1, 1 << 31, (1 << 35) + 77])
def test_grids_hold_every_workgroup(sizes, groups):
    x, y = sizes.grid_x(groups), sizes.grid_y(groups)
    assert 1 <= x and x * 1024 < 1 << 32 and 1 <= y <= 65535
    # workgroups (i, j) are numbers j row + i: each of 0 .. groups - 1 is there once, and less than a row behind them
    assert y == 1 and x == groups or x == sizes.grid_row()
    assert 0 <= x * y - groups < x


def test_tiles_of_one_launch(sizes):
    assert sizes.tiles_fit((1 << 23) - 8) and not sizes.tiles_fit((1 << 23) - 7)


@pytest.mark.parametrize("kind", [_lib.FP4Q_LINEAR, _lib.FP4Q_GATED, _lib.FP4Q_LINEAR_BACKWARD])
def test_more_tiles_than_a_launch_takes_are_refused(lib, kind):
    """2^24 tiles of 128 x 256 (a gated call's of 128 x 128): refused before anything is enqueued, not by the launch."""
    rows, out = 512, 1 << 30
    w = weight(n=out, k=16) if kind != _lib.FP4Q_LINEAR_BACKWARD else weight(n=16, k=out)
    call = (lib.fp4q_linear, lib.fp4q_gated, lib.fp4q_linear_backward)[kind]
    assert call(w, linear_args(rows=rows, x_stride=16), None, 0, None) == UNSUPPORTED
    assert lib.fp4q_linear_workspace_bytes(w, linear_args(rows=rows, x_stride=16), kind) == 0


def test_eight_bit_rows_of_the_few_row_kernel(sizes):
    """Its last element's offset stays below 2^31, and one row of any length is taken."""
    for k in (32, 4096, 1 << 20, (1 << 25) - 32, 1 << 25, (1 << 31) - 32):
        for rows in (1, 2, 16, 63, 64):
            assert bool(sizes.few_eight_fits(rows, k)) == (rows * k < 1 << 31)
    assert sizes.few_eight_fits(1, (1 << 31) - 32)
