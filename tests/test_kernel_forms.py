"""Every size that a GPU test means for one form of the kernels takes that form (the rules are host
code, compiled here)."""
import os
import shutil
import subprocess

import pytest

import form_sizes as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MODES = {"forward": 0, "dx": 1, "dw": 2, "mx": 3, "both": 4}


@pytest.fixture(scope="module")
def form_of(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("forms") / "kernel_forms")
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I/opt/rocm/include",
                    "-D__HIP_PLATFORM_AMD__", os.path.join(ROOT, "tests", "kernel_forms.cpp"), "-o", exe],
                   check=True)

    def forms(cases):
        text = "".join(f"{MODES[mode]} {rows * share} {max(groups, 1)} {int(groups > 0)} {h_in} {h_out}\n"
                       for mode, (rows, share, groups, h_in, h_out) in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60).stdout
        return [tuple(int(v) for v in line.split()) for line in out.splitlines()]

    return forms


def test_sizes_take_the_forms_they_are_meant_for(form_of):
    cases = list(F.cases())
    got = form_of([(mode, size) for mode, size, _ in cases])
    assert len(got) == len(cases)
    wrong = [(case, form) for case, form in zip(cases, got) if form != (*case[2], 1)]
    assert not wrong, wrong


def test_the_sizes_meet_every_form(form_of):
    met = {(mode, form) for mode, _, form in F.cases()}
    assert met == {("forward", F.STREAM_16), ("mx", F.STREAM_4_DEEP), ("mx", F.STREAM_4_WIDE),
                   ("both", F.STREAM_4_DEEP), ("both", F.STREAM_4_WIDE), ("mx", F.TILE_128), ("mx", F.TILE_HALF),
                   ("mx", F.TILE_256), ("both", F.TILE_128), ("both", F.TILE_256)}


def test_tiled_forms_of_16_bit_weights(form_of):
    """The sizes of test_gpu_grouped.py's test of the largest tiles."""
    sizes = [(4200, 1, 3, 200, 4096), (2300, 2, 2, 392, 4000), (4097, 1, 1, 72, 4104)]
    assert all(f == (*F.TILE_256, 1) for f in form_of([("forward", s) for s in sizes]))
    assert all(f == (*F.TILE_256, 1) for f in form_of([("dx", (r, s, g, wide, k)) for r, s, g, k, wide in sizes]))
    assert all(f == (*F.TILE_256, 1) for f in form_of([("dw", (r, s, g, wide, wide)) for r, s, g, _, wide in sizes]))
    assert form_of([("forward", (700, 1, 130, 136, 72)), ("dx", (1, 1, 1, 8, 8)), ("dw", (1, 1, 1, 8, 8))]) == \
        [(*F.TILE_128, 1)] * 3


def test_sizes_of_the_scale_tests(form_of):
    from test_gpu_mx_scales import SIZES
    got = form_of([("mx", (rows, 1, 0, h_in, h_out)) for rows, h_in, h_out in SIZES])
    assert [f[:3] for f in got] == [F.STREAM_4_DEEP] * 2 + [F.STREAM_4_WIDE] * 2 + [
        F.TILE_128, F.TILE_HALF, F.TILE_256, F.STREAM_4_DEEP, F.STREAM_4_WIDE]
    got = form_of([("both", (rows, 1, 0, h_in, h_out)) for rows, h_in, h_out in SIZES])
    assert [f[:3] for f in got[4:]] == [F.TILE_128, F.TILE_128, F.TILE_256, F.STREAM_4_DEEP, F.STREAM_4_WIDE]


def test_the_form_that_measured_faster_is_taken(form_of):
    """Both forms timed (us, streaming and tiles) where they differ by more than a tenth."""
    measured = [
        # mode, (rows, share, groups, h_in, h_out), streaming, tiles
        ("forward", (16, 1, 0, 4096, 4096), 8.9, 36.9), ("forward", (64, 1, 0, 4096, 4096), 20.6, 38.3),
        ("forward", (256, 1, 0, 4096, 4096), 68.4, 38.6), ("forward", (256, 1, 0, 8192, 1024), 36.4, 71.7),
        ("forward", (64, 1, 0, 5120, 13824), 75.4, 49.2), ("forward", (128, 1, 8, 4096, 1024), 16.6, 39.0),
        ("forward", (256, 1, 8, 5120, 13824), 347.5, 214.2), ("forward", (2048, 1, 64, 4096, 1024), 151.9, 124.9),
        ("mx", (16, 1, 0, 4096, 4096), 9.5, 44.4), ("mx", (256, 1, 0, 4096, 4096), 37.9, 44.5),
        ("mx", (512, 1, 0, 4096, 4096), 73.1, 45.6), ("mx", (512, 1, 0, 8192, 1024), 40.2, 85.0),
        ("mx", (64, 1, 0, 5120, 13824), 46.0, 55.4), ("mx", (128, 1, 0, 5120, 13824), 86.4, 56.6),
        ("mx", (1024, 1, 8, 4096, 1024), 39.6, 45.9), ("mx", (128, 1, 8, 5120, 13824), 112.7, 245.7),
        ("mx", (1024, 1, 64, 4096, 1024), 55.6, 71.5), ("mx", (2048, 1, 64, 4096, 1024), 80.0, 71.8),
        ("both", (16, 1, 0, 4096, 4096), 10.0, 13.0), ("both", (64, 1, 0, 4096, 4096), 20.1, 13.3),
        ("both", (256, 1, 0, 4096, 4096), 39.7, 13.8), ("both", (16, 1, 0, 8192, 1024), 13.7, 22.4),
        ("both", (256, 1, 0, 8192, 1024), 35.5, 23.0), ("both", (16, 1, 0, 5120, 13824), 19.2, 17.0),
        ("both", (64, 1, 0, 5120, 13824), 49.5, 18.1), ("both", (256, 1, 8, 4096, 1024), 22.2, 14.0),
        ("both", (128, 1, 8, 5120, 13824), 107.0, 92.0), ("both", (1024, 1, 64, 4096, 1024), 55.0, 27.9),
    ]
    got = form_of([(mode, size) for mode, size, _, _ in measured])
    wrong = [m for m, form in zip(measured, got) if (form[0] == F.STREAM_16[0]) != (m[2] < m[3])]
    assert not wrong, wrong
