"""The order of LDS accesses in the compiled 8-bit kernels: the streaming form's loads into a ring buffer come
after its reads have returned, and the tiled form's reads of a buffer have returned at the barrier behind which it
is filled again."""
import os
import re
import shutil
import subprocess

import pytest

from adapter_gemv_amd import build
from test_lds_order import kernels, loads_over_reads

SKINNY = """
#include "%s/sgmv_fp8_skinny.h"
using namespace sgmv_dev;
template <int DT, bool X16> void forms(const Fp8Args& A) {
  fp8_skinny_kernel<DT, X16, 1, 8><<<1, 512>>>(A);
  fp8_skinny_kernel<DT, X16, 2, 4><<<1, 256>>>(A);
}
void all_forms(const Fp8Args& A) { forms<0, false>(A); forms<0, true>(A); forms<1, false>(A); forms<1, true>(A); }
"""
TILE = """
#include "%s/sgmv_fp8_tile.h"
using namespace sgmv_dev;
void all_forms(const Fp8Args& A) {
  fp8_tile_kernel<1, false, 64, 64, 2, 2, 4, true><<<1, 256>>>(A);
  fp8_tile_kernel<1, true, 128, 128, 2, 2, 2, true><<<1, 256>>>(A);
}
"""


def listing(tmp_path, source):
    if not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")):
        pytest.skip("hipcc not found")
    (tmp_path / "k.hip").write_text(source % build.CSRC)
    subprocess.run([build._hipcc(), *build.COMMON, "--cuda-device-only", "-S", str(tmp_path / "k.hip"), "-o",
                    str(tmp_path / "k.s")], check=True, capture_output=True)
    return (tmp_path / "k.s").read_text()


def test_loads_into_the_ring_wait_for_its_reads(tmp_path):
    found = kernels(listing(tmp_path, SKINNY))
    assert len(found) == 8, sorted(found)
    for name, blocks in found.items():
        text = [t for _, b in blocks for t in b]
        assert any("load_lds" in t for t in text) and any(t.startswith("ds_read") for t in text), name
        assert not loads_over_reads(blocks), name


def test_every_barrier_of_the_tiles_waits_for_lds(tmp_path):
    """Each s_barrier stands right behind a wait for all LDS accesses."""
    text = [t.split(";")[0].strip() for t in listing(tmp_path, TILE).splitlines()]
    text = [t for t in text if t and not t.startswith(".")]
    at = [i for i, t in enumerate(text) if t == "s_barrier"]
    assert len(at) > 10
    for i in at:
        before = text[i - 1]
        assert re.match(r"s_waitcnt\b", before) and "lgkmcnt(0)" in before, text[i - 4:i + 1]


LARGE = """
#include "%%s/sgmv_fp8_tile.h"
using namespace sgmv_dev;
void all_forms(const Fp8Args& A) { fp8_tile_kernel<1, %s, 256, 256, 2, 4, 2, %s><<<1, 512>>>(A); }
"""


@pytest.mark.parametrize("dx", ["false", "true"])
@pytest.mark.parametrize("near", ["false", "true"])
def test_every_barrier_of_the_large_tiles_waits_for_all_loads(tmp_path, dx, near):
    """The same of the tiles of 256 x 256, which hold two stages: the wait before a barrier is for every load as well,
    those of spilled registers among them, so that these disturb no count."""
    text = [t.split(";")[0].strip() for t in listing(tmp_path, LARGE % (dx, near)).splitlines()]
    text = [t for t in text if t and not t.startswith(".")]
    at = [i for i, t in enumerate(text) if t == "s_barrier"]
    assert len(at) > 10
    for i in at:
        before = text[i - 1]
        assert re.match(r"s_waitcnt\b", before) and "lgkmcnt(0)" in before and "vmcnt(0)" in before, text[i - 4:i + 1]
