"""How many blocks share a sequence's verification, checked on the host (no GPU)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
VS = (1, 2047, 4096, 16384, 65535, 65536, 98304, 102400, 131072, 151936, 262144, 10 ** 7, 2 ** 31 - 2 ** 16 - 2)


@pytest.fixture(scope="module")
def blocks(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("blocks") / "harness")
    subprocess.check_call([nvcc, "-std=c++17", "-O2", "-o", exe, os.path.join(HERE, "verify_blocks_harness.cu")])

    def run(cases):
        text = "\n".join(" ".join(str(int(x)) for x in c) for c in cases)
        got = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60).stdout.split()
        return [int(x) for x in got]
    return run


def test_never_sixteen_where_the_device_runs_no_such_cluster(blocks):
    """Sixteen blocks are beyond the portable size: a device, or a part of one, that has no room for them gets eight."""
    cases = [(B, V, 0) for B in (1, 2, 12, 16, 64, 65535) for V in VS]
    got = blocks(cases)
    assert len(got) == len(cases) and set(got) <= {1, 2, 4, 8}
    assert all(n == 8 for (B, V, _), n in zip(cases, got) if V >= 65536)


def test_powers_of_two_up_to_sixteen(blocks):
    cases = [(B, V, 14) for B in (1, 2, 12, 16, 64, 65535) for V in VS]
    got = blocks(cases)
    assert len(got) == len(cases) and set(got) == {1, 2, 4, 8, 16}
    assert all(n < 16 for (B, V, _), n in zip(cases, got) if V < 98304)
