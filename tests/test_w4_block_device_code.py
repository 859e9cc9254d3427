"""What the 4-bit products' block kernels rely on in their built device code, read from the assembly that the
library's own flags give (CPU: nothing is run). A block's buffers change hands at its barriers: rows, scales and operands that
a wave has read or asked for must have arrived before it reaches one, the writes of operands (written in assembly, so
that the compiler counts no wait for them) among them."""
import os
import re
import subprocess

import pytest

pytestmark = pytest.mark.slow


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{mangled kernel name: its instructions and labels in order} of both block files."""
    from sparse_moe_routing_amd import build as lib_build
    try:
        cc = lib_build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    # -Werror off here only: hipcc adds a link flag that a device-only compile leaves unused
    flags = [f for f in lib_build.compile_flags() if f not in ("-fPIC", "-Werror")]
    runs = []
    for rows in ("bf16", "f32"):
        out = tmp_path_factory.mktemp("asm") / f"{rows}.s"
        runs.append((out, subprocess.Popen(
            [cc, *flags, "--cuda-device-only", "-S", os.path.join(lib_build.CSRC, f"w4_block_{rows}.hip"), "-o", str(out)],
            stderr=subprocess.PIPE, text=True)))
    found = {}
    for out, run in runs:
        err = run.communicate()[1]
        assert run.returncode == 0, err[-2000:]
        lines = None
        for line in out.read_text().splitlines():
            line = line.split(";")[0].strip()
            name = re.match(r"(_ZN3moe\S*w4_block_kernel\S*):$", line)
            if name:
                lines = found.setdefault(name.group(1), [])
            elif line.startswith(".Lfunc_end"):
                lines = None
            elif lines is not None and line and (not line.startswith(".") or line.startswith(".LBB")):
                lines.append(line)
    assert len(found) == 4
    return found


MEMORY = ("ds_", "buffer_", "global_", "flat_", "s_load", "s_buffer")


def unready(lines):
    """The barriers that a wave can reach with memory operations outstanding: in front of each, in the same straight
    run of code, stands a wait for all of them, and nothing that touches memory after it."""
    bad = []
    for i, line in enumerate(lines):
        if line != "s_barrier":
            continue
        loads = lds = False
        for before in reversed(lines[:i]):
            op = before.split()[0]
            if op == "s_waitcnt":
                loads = loads or "vmcnt(0)" in before
                lds = lds or "lgkmcnt(0)" in before
                if loads and lds:
                    break
            elif before.endswith(":") or op.startswith("s_cbranch") or op == "s_branch" or op.startswith(MEMORY):
                bad.append((i, before))
                break
        else:
            bad.append((i, "start"))
    return bad


def test_barriers_wait_for_everything(kernels):
    for name, lines in kernels.items():
        barriers = sum(line == "s_barrier" for line in lines)
        # four turns of a line of codes for each number of row subtiles and scale grouping, one behind the scan
        subtiles = 2 if "IfLb" in name else 3 if "Lb1E" in name else 4
        assert barriers == 1 + 2 * subtiles * 4, (name, barriers)
        bad = unready(lines)
        # the first stands behind the row tiles' scan, before any load of operands: it waits for its LDS write
        assert len(bad) <= 1, (name, bad[:4])
        if bad:
            at = bad[0][0]
            assert not any(line.startswith("buffer_load") for line in lines[:at]), (name, bad)
            assert any("lgkmcnt(0)" in line for line in lines[max(0, at - 4):at]), (name, bad)


def test_the_last_loads_are_waited_for(kernels):
    """No load into a block's LDS outlives the block."""
    for name, lines in kernels.items():
        ends = [i for i, line in enumerate(lines) if line == "s_endpgm"]
        assert ends, name
        for end in ends:
            for before in reversed(lines[:end]):
                op = before.split()[0]
                if op == "s_waitcnt" and "vmcnt(0)" in before:
                    break
                # an end that a block without units takes has loaded nothing
                assert not (op.startswith("buffer_load") and before.endswith(" lds")), (name, end, before)
