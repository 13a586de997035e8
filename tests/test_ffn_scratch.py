"""No kernel of the linear layers and the norm keeps registers in memory: what the compiler says of the code that is
built, instance by instance."""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from fp4_block_scaled_row_amd import build

SOURCES = ["fp4q_linear.hip", "fp4q_linear_few.hip", "fp4q_linear_many_mx.hip", "fp4q_linear_many_nv.hip",
           "fp4q_linear_many_back_mx.hip", "fp4q_linear_many_back_nv.hip", "fp4q_linear_mx8.hip", "fp4q_norm.hip"]


@pytest.fixture(scope="module")
def scratch(tmp_path_factory):
    """{source: {kernel: bytes of scratch a lane}}."""
    at = tmp_path_factory.mktemp("code")

    def one(source):
        out = str(at / (source + ".s"))
        r = subprocess.run([build.hipcc()] + build.FLAGS + ["--cuda-device-only", "-S", os.path.join(build.CSRC, source),
                                                            "-o", out], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return dict(re.findall(r"\.amdhsa_kernel (\S+).*?\.amdhsa_private_segment_fixed_size (\d+)", open(out).read(), re.S))

    with cf.ThreadPoolExecutor(min(8, os.cpu_count() or 4)) as pool:
        return dict(zip(SOURCES, pool.map(one, SOURCES)))


@pytest.mark.parametrize("source", SOURCES)
def test_registers_are_not_spilled(scratch, source):
    assert len(scratch[source]) >= 2
    assert {k: b for k, b in scratch[source].items() if int(b)} == {}
