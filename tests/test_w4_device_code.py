"""What the 4-bit products' streams rely on in their built device code and no result shows reliably, read
from the assembly that the library's own flags give (CPU: nothing is run)."""
import os
import re
import subprocess

import pytest

from test_operators_device_code import refills_before_reads

pytestmark = pytest.mark.slow


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{mangled kernel name: its instructions and labels in order} of w4.hip."""
    from sparse_moe_routing_amd import build as lib_build
    try:
        cc = lib_build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm") / "w4.s"
    # -Werror off here only: hipcc adds a link flag that a device-only compile leaves unused
    flags = [f for f in lib_build.compile_flags() if f not in ("-fPIC", "-Werror")]
    r = subprocess.run([cc, *flags, "--cuda-device-only", "-S", os.path.join(lib_build.CSRC, "w4.hip"), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    found, lines = {}, None
    for line in out.read_text().splitlines():
        line = line.split(";")[0].strip()
        name = re.match(r"(_ZN3moe\S*w4_stream_kernel\S*):$", line)
        if name:
            lines = found.setdefault(name.group(1), [])
        elif line.startswith(".Lfunc_end"):
            lines = None
        elif lines is not None and line and (not line.startswith(".") or line.startswith(".LBB")):
            lines.append(line)
    assert len(found) == 40
    return found


def test_refills_wait_for_the_reads_of_their_slot(kernels):
    """A slab that is loaded straight into LDS takes the place of one that has been read: the wave
    waits for those reads before it requests the load."""
    bad = {name: refills_before_reads(lines) for name, lines in kernels.items()}
    bad = {name: at[:3] for name, at in bad.items() if at}
    assert not bad, bad


def test_split_blocks_take_one_unit(kernels):
    """Where the waves of a block split K there are no more units than blocks: the waves meet once,
    to join their sums, and no loop carries them on to another unit."""
    split = {name: lines for name, lines in kernels.items() if re.search(r"Li8ELb[01]EEEv", name)}
    assert len(split) == 20
    assert {sum(line == "s_barrier" for line in lines) for lines in split.values()} == {1}
