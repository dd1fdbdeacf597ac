"""The angle's integer arithmetic, compiled for the host, against exact integers: as many answers as questions, from a program
that ended well."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from hybrid_linear_attention_conv_gb300 import build as gbuild

MAIN = r"""
#include <cstdio>
#include "gdn_rotary.cuh"
int main() {
    unsigned long long turns;
    int pos, n = 0;
    for (; scanf("%llu %d", &turns, &pos) == 2; ++n) printf("%d\n", (int)gdn::turn_fraction(turns, pos));
    return n > 0 ? 0 : 1;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    at = tmp_path_factory.mktemp("angle")
    (at / "angle.cu").write_text(MAIN)
    r = subprocess.run([nvcc, "-std=c++17", *gbuild.ARCH, "-I", gbuild.CSRC, str(at / "angle.cu"), "-o", str(at / "angle")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return str(at / "angle")


@pytest.mark.parametrize("seed", range(4))
def test_every_fraction(program, seed):
    rng = np.random.default_rng(seed)
    ends = [0, 1, -1, 2, -2, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 1 - 2 ** 31]
    pairs = [(t, p) for t in (0, 1, 2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 62, 2 ** 62 - 1) for p in ends]
    pairs += [(int(t), int(p)) for t, p in zip(rng.integers(0, 2 ** 62, 500), rng.integers(-2 ** 31, 2 ** 31, 500))]
    r = subprocess.run([program], input="\n".join(f"{t} {p}" for t, p in pairs), capture_output=True, text=True, timeout=60)
    assert r.returncode == 0
    got = [int(x) for x in r.stdout.split()]
    assert len(got) == len(pairs)
    for x, (t, p) in zip(got, pairs):
        exact = (t * p + 2 ** 31 >> 32) % 2 ** 32  # the fraction of a turn, to the nearest of 2^-32
        assert -2 ** 31 <= x < 2 ** 31 and x % 2 ** 32 == exact, (t, p)
