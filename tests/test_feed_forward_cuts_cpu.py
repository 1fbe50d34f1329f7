"""Which tiles and splits the feed-forward tests' sizes get (a C++ program, on the
CPU), so that a change of the cost model shows where a test stops running what it
is for.
"""
import os
import shutil
import subprocess

import pytest

from tests.test_gpu_feed_forward_large_tiles import BACKWARD, FORWARD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def cuts(tmp_path_factory):
    if shutil.which("hipcc") is None:
        pytest.skip("needs hipcc")
    exe = str(tmp_path_factory.mktemp("cuts") / "cuts_check")
    subprocess.run(["hipcc", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "diffusion_transformer_qk_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c_abi", "cuts_check.cpp"), "-o", exe], check=True)

    def of(rows, hidden, inner, size=2):
        """(side, tiles, splits) of the forward product, dx and dw, and the terms of dgate and dup."""
        out = subprocess.run([exe], input="%d %d %d %d\n" % (rows, hidden, inner, size), capture_output=True, text=True,
                             check=True, timeout=60).stdout
        v = [int(n) for n in out.split()]
        return [tuple(v[i:i + 3]) for i in (0, 3, 6)] + [v[9]]

    return of


def test_sizes_of_several_rounds_of_large_tiles(cuts):
    for rows, hidden, inner in FORWARD:
        for size, unit in ((2, 8), (1, 16)):
            side, tiles, _ = cuts(rows, unit * -(-hidden // unit), unit * -(-inner // unit), size)[0]
            assert side == 256 and tiles > 512, (rows, hidden, inner, size)
            assert rows % 256 and inner % 128
    (side, tiles, splits), at = cuts(*BACKWARD[0])[1], BACKWARD[0]
    assert (side, splits) == (256, 1) and tiles > 512 and at[0] % 256 and at[1] % 256
    (side, tiles, splits), at = cuts(*BACKWARD[1])[2], BACKWARD[1]
    assert (side, splits) == (256, 1) and tiles > 512 and at[1] % 256 and at[2] % 256


@pytest.mark.parametrize("size,forward,dx,dw", [
    # several rounds of small tiles
    ((4200, 96, 2056), 128, None, None), ((257, 200, 16392), 128, None, None), ((5000, 104, 1800), 128, None, None),
    ((4200, 4104, 72), None, (128, 1), None), ((136, 2056, 4104), None, None, (128, 1)),
    # one round of large ones, with splits and without
    ((3900, 96, 1960), 256, None, None), ((300, 200, 16328), 256, None, None), ((520, 1040, 8008), 256, None, None),
    ((3900, 3920, 72), None, (256, 1), None), ((136, 3920, 1960), None, None, (256, 1)),
    # few rows, and splits of small tiles
    ((5, 512, 2048), 128, (128, True), None), ((2500, 64, 136), None, None, (128, True)),
    ((3000, 520, 40), None, None, (128, True)), ((40, 264, 3080), None, (128, True), None),
    # workloads: a video latent, an image, their gradients
    ((32760, 5120, 13824), 256, None, None), ((4608, 6144, 16384), 256, (256, 1), (256, 1)),
    ((256, 5120, 13824), 128, None, None),
])
def test_sizes_of_other_tests(cuts, size, forward, dx, dw):
    found = cuts(*size)
    if forward:
        assert found[0][0] == forward and found[0][2] == 1
    for want, got in ((dx, found[1]), (dw, found[2])):
        if want:
            assert got[0] == want[0]
            assert got[2] > 1 if want[1] is True else got[2] == want[1]


def test_terms(cuts):
    """Two for up to 32 rows, and for 2^15 numbers of up to 2^20 of x."""
    for size in ((1, 5120, 13824), (32, 8192, 16384), (33, 8, 992), (128, 8192, 256), (4096, 256, 8)):
        assert cuts(*size)[3] == 2, size
    for size in ((33, 5120, 13824), (33, 8, 1000), (129, 8192, 248), (4096, 264, 8), (4104, 8, 8), (32760, 40, 8),
                 (4608, 6144, 16384)):
        assert cuts(*size)[3] == 1, size
