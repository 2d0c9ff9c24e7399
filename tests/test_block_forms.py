"""Every size that a GPU test means for one form of the 8-bit products takes that form (the rules are host code,
compiled here), the forms that measured faster are taken, and workspaces are asked for where they are used."""
import os
import shutil
import subprocess

import pytest

import block_sizes as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def form_of(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("forms") / "block_forms")
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__",
                    os.path.join(ROOT, "tests", "block_forms.cpp"), "-o", exe], check=True)

    def forms(cases):
        text = ""
        for dx, (rows, share, groups, depth, out) in cases:
            h_in, h_out = (out, depth) if dx else (depth, out)
            text += f"{int(dx)} {rows * share} {max(groups, 1)} {int(groups > 0)} {h_in} {h_out}\n"
        done = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60).stdout
        return [tuple(int(v) for v in line.split()) for line in done.splitlines()]

    return forms


def test_sizes_take_the_forms_they_are_meant_for(form_of):
    cases = list(F.cases())
    got = form_of([(dx, size) for dx, size, _ in cases])
    wrong = [(case, form) for case, form in zip(cases, got) if form != (*case[2], 1)]
    assert len(got) == len(cases) and not wrong, "\n".join(map(str, wrong))


def test_the_form_that_measured_faster_is_taken(form_of):
    """us of streaming and of tiles of 64, 128 and 256 where the best is ahead by more than a tenth."""
    measured = [
        ((32, 1, 0, 2048, 2048), 9.4, 12.2, 16.1, None), ((64, 1, 0, 4096, 4096), 20.3, 22.8, 29.9, None),
        ((256, 1, 0, 4096, 4096), 44.8, 23.7, 34.9, None), ((1024, 1, 0, 4096, 4096), 152, 50.7, 38.1, None),
        ((16, 1, 0, 5120, 13824), 26.1, 31.1, 43.4, None), ((64, 1, 0, 5120, 13824), 56.9, 32.4, 40.0, None),
        ((256, 1, 0, 5120, 13824), 168, 70.2, 45.0, None), ((128, 1, 0, 8192, 1024), 21.4, 32.9, 55.7, None),
        ((2048, 1, 64, 4096, 1024), 116, 78.8, 85.6, None), ((512, 1, 8, 5120, 13824), 359, 190, 152, None),
        ((8192, 1, 0, 8192, 8192), None, 1090, None, 541),
    ]
    for size, *times in measured:
        best = min((t, i) for i, t in enumerate(times) if t is not None)[1]
        assert form_of([(False, size)])[0][0] == (32, 64, 128, 256)[best], size


def test_workspace_follows_the_form():
    from adapter_gemv_amd import _lib
    call = _lib.lib().sgmv_block_workspace_bytes
    for form, sizes in F.FORWARD.items():
        for rows, share, groups, depth, out in sizes:
            room = call(rows * share, share, max(groups, 1), int(groups > 0), depth, out)
            want = (rows * depth + 255) // 256 * 256 + rows * -(-depth // 128) * 4
            assert room == (0 if form[3] == 0 else want), (form, rows, depth, out)
