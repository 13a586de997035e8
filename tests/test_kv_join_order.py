"""The order that joining a context's pieces rests on, in the code that is built: a workgroup's stores of its piece have
completed, in every wave (a wait for all of them, then a barrier), before its arrival is counted."""
import os
import re
import subprocess

import pytest

from fp4_block_scaled_row_amd import build


@pytest.mark.parametrize("source", ["fp4q_kv_decode_nv64.hip", "fp4q_kv_decode_mx128.hip"])
def test_arrivals_are_counted_after_the_stores(source, tmp_path):
    out = str(tmp_path / "kernels.s")
    r = subprocess.run([build.hipcc()] + build.FLAGS + ["--cuda-device-only", "-S", os.path.join(build.CSRC, source), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    kernels = open(out).read().split(".amdhsa_kernel")
    counted = 0
    for text in kernels:
        code = [line.strip() for line in text.splitlines()]
        for at, line in enumerate(code):
            if not line.startswith("global_atomic_add"):
                continue
            counted += 1
            # back to the barrier before the count: no store between; then the wait, before any store
            back = at
            while not code[back].startswith("s_barrier"):
                assert "_store_" not in code[back] or code[back].startswith(("ds_", "scratch_")), code[back]
                back -= 1
            while not re.match(r"s_waitcnt .*vmcnt\(0\)", code[back]):
                assert not code[back].startswith(("global_store", "flat_store", "buffer_store")), code[back]
                back -= 1
    assert counted >= 4
