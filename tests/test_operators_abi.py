"""The separate operators' refusals, on the CPU: every bad call returns its status before anything
is enqueued (the addresses below are never dereferenced), and the binding's checks raise."""
import ctypes

import pytest

from sparse_moe_routing_amd import binding
from sparse_moe_routing_amd.binding import (MOE_BF16, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED,
                                            MOE_F32, MOE_FP8_E4M3, MOE_OK)

A = 0x10000000  # 16-byte aligned, never read
INV, UNS = MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return binding.load()


# argument order of each entry point, with values of a good call
GOOD = {
    "moe_permute": dict(x=A, rows=A, T=4, H=64, n_rows=32, dtype=MOE_BF16, xs=A, s=None),
    "moe_permute_backward": dict(dxs=A, rows=A, T=4, H=64, n_rows=32, dtype=MOE_F32, dx=A, s=None),
    "moe_unpermute": dict(ys=A, rows=A, w=A, shared=A, gate=A, T=4, H=64, n_rows=32,
                          dtype=MOE_BF16, y=A, y_dtype=MOE_F32, s=None),
    "moe_unpermute_backward": dict(dy=A, ys=A, rows=A, w=A, shared=A, gate=A, T=4, H=64,
                                   n_rows=32, dtype=MOE_BF16, y_dtype=MOE_F32, dys=A, dw=A,
                                   dshared=A, dgate=A, s=None),
    "moe_quantize_i8": dict(x=A, n=4, K=64, dtype=MOE_F32, q=A, scale=A, s=None),
    "moe_permute_i8": dict(x=A, rows=A, T=4, H=64, n_rows=32, dtype=MOE_BF16, xs=A, xs_scale=A,
                           s=None),
    "moe_matmul_i8": dict(x=A, x_scale=A, n_rows=4, w=A, w_scale=A, E=2, M=64, K=64, offsets=A,
                          swiglu=0, y=A, y_dtype=MOE_BF16, s=None),
}
POINTERS16 = {"x", "xs", "dxs", "dx", "ys", "y", "dy", "dys", "q", "shared", "dshared"}
POINTERS4 = {"rows", "gate", "dw", "dgate", "scale", "xs_scale", "x_scale", "w_scale", "offsets"}
OPTIONAL = {"offsets"}


def call(lib, name, **changed):
    args = dict(GOOD[name], **changed)
    return getattr(lib, name)(*args.values())


def bad_calls():
    for name, good in GOOD.items():
        for arg in good:
            if arg in POINTERS16 or (arg == "w" and name == "moe_matmul_i8"):
                yield name, {arg: A + 8}, INV
                yield name, {arg: None}, INV
            if arg in POINTERS4 or (arg == "w" and name != "moe_matmul_i8"):
                yield name, {arg: A + 2}, INV
                yield name, {arg: None}, INV  # offsets NULL: with E = 2
            if arg in ("dtype", "y_dtype"):
                for d in (MOE_FP8_E4M3, 7, -1):
                    yield name, {arg: d}, INV
            if arg in ("T", "n", "n_rows"):
                yield name, {arg: -1}, INV
                yield name, {arg: 8388609}, UNS
            if arg == "T":
                yield name, {arg: 1048577}, UNS
            if arg in ("H", "K"):
                step = 16 if name.endswith("i8") else 8
                for v in (0, -step, step // 2, 64 + step // 2, 16384 + step):
                    yield name, {arg: v}, UNS
    for kw, want in (({"E": 0}, UNS), ({"E": 257}, UNS), ({"M": 0}, UNS), ({"M": 60}, UNS),
                     ({"M": 65544}, UNS), ({"M": 72, "swiglu": 1}, UNS), ({"swiglu": 2}, INV),
                     ({"swiglu": -1}, INV)):
        yield "moe_matmul_i8", kw, want


@pytest.mark.parametrize("name,changed,want", list(bad_calls()),
                         ids=lambda v: v if isinstance(v, str) else str(v))
def test_refused(lib, name, changed, want):
    assert call(lib, name, **changed) == want


@pytest.mark.parametrize("name", list(GOOD))
def test_nothing_to_do(lib, name):
    """No tokens, or no rows: fine, with nothing enqueued and no pointer needed."""
    count = "n" if "n" in GOOD[name] else "T" if "T" in GOOD[name] else "n_rows"
    none = {a: None for a in GOOD[name] if a in POINTERS16 | POINTERS4 | {"w"} and a != "offsets"}
    assert call(lib, name, **{count: 0}, **none) == MOE_OK
    if name in ("moe_permute", "moe_permute_i8"):  # every pair dropped
        assert call(lib, name, n_rows=0) == MOE_OK


OUTPUTS = {"moe_permute": ["xs"], "moe_permute_backward": ["dx"], "moe_unpermute": ["y"],
           "moe_unpermute_backward": ["dys", "dw", "dshared", "dgate"],
           "moe_quantize_i8": ["q", "scale"], "moe_permute_i8": ["xs", "xs_scale"],
           "moe_matmul_i8": ["y"]}


def overlaps():
    for name, outs in OUTPUTS.items():
        for out in outs:
            for arg in GOOD[name]:
                if arg != out and (arg in POINTERS16 | POINTERS4 or arg == "w"):
                    yield name, out, arg


@pytest.mark.parametrize("name,out,other", list(overlaps()))
def test_overlap_refused(lib, name, out, other):
    """An output that shares memory with another operand, from either side: every operand has a
    place of its own, 16 MiB apart, but for the two. (The smallest operand takes 12 bytes.)"""
    places = {a: A + (i << 24) for i, a in enumerate(GOOD[name])
              if a in POINTERS16 | POINTERS4 or a == "w"}
    last4 = 8 if out in POINTERS4 or other in POINTERS4 else 0
    assert call(lib, name, **dict(places, **{out: places[other]})) == INV
    if other in POINTERS4 or (other == "w" and name != "moe_matmul_i8"):
        assert call(lib, name, **dict(places, **{other: places[out] + last4})) == INV
    elif out in POINTERS4:
        assert call(lib, name, **dict(places, **{out: places[other] + last4})) == INV


def test_shared_arguments_come_together(lib):
    for name in ("moe_unpermute", "moe_unpermute_backward"):
        opt = [a for a in ("shared", "gate", "dshared", "dgate") if a in GOOD[name]]
        for a in opt:
            assert call(lib, name, **{b: None for b in opt if b != a}) == INV


def test_bucket_rows_refuses(lib):
    assert lib.moe_bucket_rows(None, A, 4, A, A, A, A, A, 1 << 20, None) == INV


def test_binding_checks_tensors():
    """Wrong dtypes, shapes, strides and devices raise before the library is called."""
    import torch
    x = torch.zeros(4, 64)
    rows = torch.zeros(32, dtype=torch.int32)
    w = torch.ones(4, 8)
    cases = [
        lambda: binding.permute(x, rows),  # not on a GPU
        lambda: binding.permute(x.half(), rows),
        lambda: binding.permute(x, rows.long()),
        lambda: binding.permute(x, rows[:24]),
        lambda: binding.permute(x.t().contiguous().t(), rows),
        lambda: binding.permute(x[:, :, None], rows),
        lambda: binding.permute_backward(torch.zeros(32, 64), rows),
        lambda: binding.unpermute(torch.zeros(32, 64), rows, w.double()),
        lambda: binding.unpermute(torch.zeros(32, 64), rows, w, shared=x),
        lambda: binding.unpermute(torch.zeros(32, 64), rows, w, gate=w[:, 0].contiguous()),
        lambda: binding.unpermute_backward(x, torch.zeros(32, 63), rows, w),
        lambda: binding.quantize_i8(x),
        lambda: binding.quantize_i8(x.to(torch.int32)),
        lambda: binding.permute_i8(x, rows[1:]),
        lambda: binding.matmul_i8(x.to(torch.int8), w[:, 0].contiguous(),
                                  torch.zeros(1, 64, 32, dtype=torch.int8), torch.ones(1, 64)),
        lambda: binding.matmul_i8(x.to(torch.int8), torch.ones(4),
                                  torch.zeros(2, 64, 64, dtype=torch.int8), torch.ones(2, 64),
                                  offsets=torch.zeros(2, dtype=torch.int32)),
    ]
    for i, f in enumerate(cases):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was not refused")
