"""How many blocks share a sequence's verification, checked on the host (no GPU)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
VS = (1, 2047, 4096, 16384, 65535, 65536, 98304, 102400, 131072, 151936, 262144, 10 ** 7, 2 ** 31 - 2 ** 16 - 2)

KINDS = [(size, draft, automaton) for size in (2, 4) for draft in (0, 1) for automaton in (0, 1)]


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
    cases = [(B, V, *kind, 0) for kind in KINDS for B in (1, 2, 12, 16, 64, 65535) for V in VS]
    got = blocks(cases)
    assert len(got) == len(cases) and set(got) <= {1, 2, 4, 8}
    assert all(n == 8 for (B, V, *_), n in zip(cases, got) if V >= 65536)


def test_powers_of_two_up_to_sixteen(blocks):
    cases = [(B, V, *kind, 14) for kind in KINDS for B in (1, 2, 12, 16, 64, 65535) for V in VS]
    got = blocks(cases)
    assert len(got) == len(cases) and set(got) == {1, 2, 4, 8, 16}
    assert all(n < 16 for (B, V, *_), n in zip(cases, got) if V < 98304)


# (sequences, V, bytes of an element, draft, automaton, us with eight blocks, with sixteen)
MEASURED = [
    (8, 65536, 2, 1, 1, 34.8, 36.8), (8, 98304, 2, 1, 1, 53.4, 43.9), (8, 151936, 2, 1, 1, 46.4, 37.0), (16, 262144, 2, 1, 1, 80.0, 63.7),
    (24, 131072, 2, 1, 1, 45.2, 53.5), (8, 98304, 4, 0, 1, 22.6, 20.5), (8, 151936, 4, 0, 1, 37.0, 30.8), (18, 106496, 4, 0, 1, 30.9, 34.9),
    (8, 65536, 2, 0, 1, 26.6, 26.7), (8, 151936, 2, 0, 1, 37.0, 28.8), (16, 151936, 2, 0, 1, 36.9, 30.8), (15, 98304, 2, 0, 1, 26.7, 34.8),
    (24, 114688, 2, 0, 1, 26.6, 36.5), (8, 65536, 2, 1, 0, 26.7, 29.5), (8, 98304, 2, 1, 0, 35.0, 32.9), (12, 102400, 2, 1, 0, 36.9, 32.8),
    (16, 131072, 2, 1, 0, 40.2, 42.7), (13, 98304, 4, 1, 0, 28.8, 32.8), (11, 114688, 4, 1, 0, 30.7, 32.6), (8, 131072, 4, 1, 0, 34.5, 28.8),
    (14, 131072, 4, 1, 0, 34.9, 32.8), (15, 131072, 4, 1, 0, 34.9, 41.9), (4, 262144, 4, 1, 0, 45.2, 36.9), (8, 65536, 4, 0, 0, 14.4, 16.4),
    (4, 262144, 4, 0, 0, 20.5, 16.7), (16, 131072, 4, 0, 0, 16.5, 20.6), (10, 98304, 2, 0, 0, 20.7, 22.7), (8, 131072, 2, 0, 0, 18.5, 20.5),
    (10, 151936, 2, 0, 0, 18.5, 16.5), (8, 200000, 2, 0, 0, 26.6, 22.6),
]


def test_the_faster_number_by_what_was_measured(blocks):
    got = blocks([c[:5] + (14,) for c in MEASURED])
    for (*case, eight, sixteen), n in zip(MEASURED, got):
        assert (sixteen if n == 16 else eight) <= 1.01 * min(eight, sixteen), case
