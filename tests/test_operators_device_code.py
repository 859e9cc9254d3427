"""What the 8-bit integer products rely on in their built device code and no result shows
reliably, read from the assembly that the library's own flags give (CPU: nothing is run)."""
import os
import re
import subprocess

import pytest

pytestmark = pytest.mark.slow


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{mangled kernel name: its instructions and labels in order} of int8.hip."""
    from sparse_moe_routing_amd import build as lib_build
    try:
        cc = lib_build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm") / "int8.s"
    # -Werror off here only: hipcc adds a link flag that a device-only compile leaves unused
    flags = [f for f in lib_build.compile_flags() if f not in ("-fPIC", "-Werror")]
    r = subprocess.run([cc, *flags, "--cuda-device-only", "-S",
                        os.path.join(lib_build.CSRC, "int8.hip"), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    found, lines = {}, None
    for line in out.read_text().splitlines():
        line = line.split(";")[0].strip()
        name = re.match(r"(_ZN3moe\S*kernel\S*):$", line)
        if name:
            lines = found.setdefault(name.group(1), [])
        elif line.startswith(".Lfunc_end"):
            lines = None
        elif lines is not None and line and (not line.startswith(".") or line.startswith(".LBB")):
            lines.append(line)
    assert len(found) == 32  # 16 block forms, 16 stream forms
    return found


def refills_before_reads(lines):
    """The loads into LDS that some path issues while LDS reads of the wave may be outstanding. The
    counter that a wait names holds LDS reads and writes, which finish in order; scalar loads
    count there too but finish in any order, so with one of them only a wait for zero tells."""
    blocks, label = {}, "entry"
    order = [label]
    for line in lines:
        if line.endswith(":"):
            label = line[:-1]
            order.append(label)
        else:
            blocks.setdefault(label, []).append(line)
    pending = {"entry": []}
    bad, work = set(), ["entry"]
    while work:
        label = work.pop()
        q, ends = list(pending[label]), False

        def reach(target):
            if target not in pending or len(q) > len(pending[target]):
                pending[target] = list(q)
                work.append(target)

        for i, line in enumerate(blocks.get(label, [])):
            op = line.split()[0]
            if op.startswith("ds_"):
                q.append("read" if "read" in op else "lds")
            elif op.startswith("s_load") or op.startswith("s_buffer_load"):
                q.append("scalar")
            elif op == "s_waitcnt":
                n = re.search(r"lgkmcnt\((\d+)\)", line)
                if n and int(n.group(1)) == 0:
                    q = []
                elif n and "scalar" not in q:
                    q = q[max(0, len(q) - int(n.group(1))):]
            elif op.startswith("buffer_load") and line.endswith(" lds"):
                if "read" in q:
                    bad.add((label, i, line))
            elif op.startswith("s_cbranch"):
                reach(line.split()[1])
            elif op == "s_branch":
                reach(line.split()[1])
                ends = True
                break
            elif op == "s_endpgm":
                ends = True
                break
        if not ends and order.index(label) + 1 < len(order):
            reach(order[order.index(label) + 1])
    return sorted(bad)


def test_refills_wait_for_the_reads_of_their_slot(kernels):
    """A slab that is loaded straight into LDS takes the place of one that has been read: the wave
    waits for those reads before it requests the load. Not asked of the block kernel's deep form
    (its last template argument true): it reads a unit's scales, which no slab overwrites, next to
    the request of the unit's third slab; its slabs are read and refilled on two sides of a
    barrier that waits for the reads."""
    forms = {name: lines for name, lines in kernels.items() if "ELb1EEEvNS" not in name}
    assert len(forms) == 24
    bad = {name: refills_before_reads(lines) for name, lines in forms.items()}
    bad = {name: at for name, at in bad.items() if at}
    assert not bad, {name: at[:3] for name, at in bad.items()}


def test_the_scan_sees_an_early_refill():
    """The check itself, on a short listing: the reads of the loop's turn are waited for in part."""
    listing = ["s_load_dwordx4 s[0:3], s[4:5], 0x0", "s_waitcnt lgkmcnt(0)", ".LBB0_1:",
               "s_waitcnt vmcnt(4)", "ds_read_b128 v[0:3], v9", "ds_read_b128 v[4:7], v9 offset:64",
               "s_waitcnt lgkmcnt(1)", "buffer_load_dwordx4 v8, s[0:3], 0 offen lds",
               "s_waitcnt lgkmcnt(0)", "buffer_load_dwordx4 v8, s[0:3], 0 offen offset:16 lds",
               "s_cbranch_scc1 .LBB0_1", "s_endpgm"]
    early = refills_before_reads(listing)
    assert [line for _, _, line in early] == ["buffer_load_dwordx4 v8, s[0:3], 0 offen lds"]
    del listing[7]
    assert refills_before_reads(listing) == []


def test_split_blocks_take_one_unit(kernels):
    """Where the waves of a block split K there are no more units than blocks: the waves meet once,
    to join their sums, and no loop carries them on to another unit."""
    split = {name: lines for name, lines in kernels.items() if re.search(r"stream.*Li4EEEv", name)}
    assert len(split) == 8
    assert {sum(line == "s_barrier" for line in lines) for lines in split.values()} == {1}
