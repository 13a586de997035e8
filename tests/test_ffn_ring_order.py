"""The order that the rings of LDS buffers rest on, in the code that is built: before each meeting of a workgroup's waves
every wave has waited for its part of the stage that is multiplied next, and for its own writes to LDS.

A step asks for one stage after its barrier.  The wait before the next barrier leaves at most N loads on their way; with
N or more of them asked for since the last barrier, everything that was asked for before that barrier has arrived: the
stage after the last one among it."""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from fp4_block_scaled_row_amd import build

SOURCES = ["fp4q_linear_many_mx.hip", "fp4q_linear_many_nv.hip", "fp4q_linear_many_back_mx.hip",
           "fp4q_linear_many_back_nv.hip", "fp4q_linear_mx8.hip"]
LOAD = re.compile(r"(global|buffer|flat)_load")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{source: {kernel: its instructions}} of the ring kernels."""
    at = tmp_path_factory.mktemp("code")

    def one(source):
        out = str(at / (source + ".s"))
        r = subprocess.run([build.hipcc()] + build.FLAGS + ["--cuda-device-only", "-S", os.path.join(build.CSRC, source),
                                                            "-o", out], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        found = {}
        for name, body in re.findall(r"^(_Z\S+):\s*;.*?\n(.*?)^\.Lfunc_end", open(out).read(), re.S | re.M):
            if "ring_kernel" in name or "mx8_kernel" in name:
                lines = [line.split(";")[0].strip() for line in body.splitlines()]
                found[name] = [line for line in lines if line and not line.startswith(".")]
        return found

    with cf.ThreadPoolExecutor(min(8, os.cpu_count() or 4)) as pool:
        return dict(zip(SOURCES, pool.map(one, SOURCES)))


def left(line):
    """Loads that a wait leaves on their way, or None where it waits for none."""
    m = re.match(r"s_waitcnt .*?vmcnt\((\d+)\)", line)
    return int(m[1]) if m else None


@pytest.mark.parametrize("source", SOURCES)
def test_stages_have_arrived_where_waves_meet(kernels, source):
    assert kernels[source]
    for name, code in kernels[source].items():
        into_lds = [i for i, line in enumerate(code) if line.startswith("buffer_load") and line.endswith("lds")]
        barriers = [i for i, line in enumerate(code) if line.startswith("s_barrier")]
        steps = [i for i in barriers if i > into_lds[0]][:sum(i < into_lds[-1] for i in barriers if i > into_lds[0])]
        assert len(steps) == 5, name                   # three of the loop and two behind it
        stage = sum(steps[0] < i < steps[1] for i in into_lds)
        assert sum(i < steps[0] for i in into_lds) == 2 * stage, name
        for n, at in enumerate(steps):
            # the nearest wait before the barrier, with no load between; it is for this wave's LDS accesses as well
            wait = at - 1
            while left(code[wait]) is None:
                assert not LOAD.match(code[wait]) and not code[wait].startswith("ds_"), (name, n, code[wait])
                wait -= 1
            assert "lgkmcnt(0)" in code[wait], (name, n)
            # (the first: since the first stage's last load)
            since = steps[n - 1] if n else [i for i in into_lds if i < at][stage - 1]
            asked = sum(bool(LOAD.match(line)) for line in code[since + 1:wait])
            assert stage <= asked and left(code[wait]) <= asked, (name, n, asked, code[wait])
            # and this step's stage goes into LDS behind the barrier alone
            assert sum(at < i < (steps[n + 1] if n < 4 else len(code)) for i in into_lds) == stage, (name, n)
