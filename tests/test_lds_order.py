"""The order of LDS accesses in the compiled streaming kernels, read from the compiler's own
listing of them.

A wavefront's ring buffer is filled again by loads that go straight into LDS, and the hardware
does not hold such a load back for LDS reads that are still in flight: between a read and the
next load into LDS there has to be a wait for the read."""
import os
import re
import shutil
import subprocess

import pytest

from adapter_gemv_amd import build

SOURCE = """
#include "%s/sgmv_skinny.h"
using namespace sgmv_dev;
hipError_t all_forms(int32_t t, hipStream_t s, const SkinnyArgs& A) {
  hipError_t e = launch_skinny<false, false>(t, s, A);
  if (e == hipSuccess) e = launch_skinny<true, false>(t, s, A);
  return e == hipSuccess ? launch_skinny<true, true>(t, s, A) : e;
}
"""


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    if not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")):
        pytest.skip("hipcc not found")
    at = tmp_path_factory.mktemp("listing")
    (at / "skinny.hip").write_text(SOURCE % build.CSRC)
    subprocess.run([build._hipcc(), *build.COMMON, "--cuda-device-only", "-S", str(at / "skinny.hip"),
                    "-o", str(at / "skinny.s")], check=True, capture_output=True)
    return (at / "skinny.s").read_text()


def kernels(listing):
    """{name: [(label, instructions)]} of the kernels in a listing."""
    out, name = {}, None
    for line in listing.splitlines():
        text = line.split(";")[0].strip()
        start = re.match(r"(_Z\w*skinny_kernel\w*):", text)
        if start:
            name = start.group(1)
            out[name] = [("", [])]
        elif text.startswith(".Lfunc_end"):
            name = None
        elif name and re.match(r"\.LBB\w+:", text):
            out[name].append((text[:-1], []))
        elif name and text:
            out[name][-1][1].append(text)
    return out


def loads_over_reads(blocks):
    """The loads into LDS that some path reaches while an LDS read is in flight."""
    index = {label: i for i, (label, _) in enumerate(blocks)}
    found, seen, todo = set(), set(), [(0, ())]
    while todo:
        at, queue = todo.pop()           # queue: whether each LDS access in flight is a read
        if (at, queue) in seen or at >= len(blocks):
            continue
        seen.add((at, queue))
        for text in blocks[at][1]:
            op = text.split()[0]
            if op.startswith("ds_"):
                queue = (*queue, op.startswith("ds_read"))[-16:]
            elif op == "s_waitcnt" and "lgkmcnt" in text:
                left = int(re.search(r"lgkmcnt\((\d+)\)", text).group(1))
                queue = queue[max(len(queue) - left, 0):]
            elif "load_lds" in op and any(queue):
                found.add(text)
            elif op.startswith("s_cbranch") or op == "s_branch":
                todo.append((index[text.split()[1]], queue))
            if op in ("s_branch", "s_endpgm"):
                break
        else:
            todo.append((at + 1, queue))
    return found


def test_loads_into_the_ring_wait_for_its_reads(listing):
    found = kernels(listing)
    assert len(found) == 10, sorted(found)
    for name, blocks in found.items():
        text = [t for _, b in blocks for t in b]
        assert any("load_lds" in t for t in text) and any(t.startswith("ds_read") for t in text), name
        assert not loads_over_reads(blocks), name


def test_a_missing_wait_is_found():
    code = [("", ["ds_read_b128 v[0:3], v9", "s_cbranch_execz .LBB0_2"]),
            (".LBB0_1", ["s_waitcnt lgkmcnt(0)"]), (".LBB0_2", ["global_load_lds_dwordx4 v[4:5], off", "s_endpgm"])]
    assert loads_over_reads(code)
    code[0][1].insert(1, "s_waitcnt vmcnt(3) lgkmcnt(0)")
    assert not loads_over_reads(code)
    code[0][1][1] = "s_waitcnt lgkmcnt(1)"
    assert loads_over_reads(code)
