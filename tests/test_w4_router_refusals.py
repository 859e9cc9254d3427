"""Refusals of the 4-bit products and of the router's training operators, on the CPU: every bad call of the
ABI returns its status before anything is enqueued (the addresses below are never dereferenced),
and the binding's checks raise before the library is called."""
import pytest

from sparse_moe_routing_amd import binding
from sparse_moe_routing_amd.binding import (MOE_BF16, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED,
                                            MOE_ERR_WORKSPACE, MOE_F32, MOE_FP8_E4M3, MOE_OK)

A = 0x10000000  # 16-byte aligned, never read
INV, UNS = MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return binding.load()


# argument order of each entry point, with values of a good call
GOOD = {
    "moe_matmul_w4": dict(x=A, n_rows=4, dtype=MOE_BF16, w=A, scale=A, scale_dtype=MOE_BF16, zero=A,
                          E=2, M=64, K=128, group=64, offsets=A, swiglu=0, y=A, y_dtype=MOE_BF16,
                          s=None),
    "moe_balance_loss": dict(logits=A, ids=A, mask=A, T=4, E=64, R=65, dtype=MOE_F32, loss=A,
                             counts=A, tokens=A, ws=A, ws_bytes=1 << 20, s=None),
    "moe_balance_loss_backward": dict(dloss=A, logits=A, counts=A, tokens=A, mask=A, T=4, E=64, R=65,
                                      dtype=MOE_F32, dlogits=A, s=None),
    "moe_route_backward": dict(dw=A, w=A, ids=A, dgate=A, gate=A, T=4, E=64, dlogits=A, s=None),
}
ALIGN = {"moe_matmul_w4": dict(x=16, w=16, scale=16, zero=16, offsets=4, y=16),
         "moe_balance_loss": dict(logits=4, ids=4, loss=4, counts=4, tokens=4),
         "moe_balance_loss_backward": dict(dloss=4, logits=4, counts=4, tokens=4, dlogits=4),
         "moe_route_backward": dict(dw=4, w=4, ids=4, dgate=4, gate=4, dlogits=16)}
OUTPUTS = {"moe_matmul_w4": ["y"], "moe_balance_loss": ["loss", "counts", "tokens"],
           "moe_balance_loss_backward": ["dlogits"], "moe_route_backward": ["dlogits"]}
MAY_BE_NULL = {"zero", "mask"}


def call(lib, name, **changed):
    args = dict(GOOD[name], **changed)
    return getattr(lib, name)(*args.values())


def bad_calls():
    for name, pointers in ALIGN.items():
        for arg, a in pointers.items():
            yield name, {arg: A + a // 2}, INV
            if arg not in MAY_BE_NULL:
                yield name, {arg: None}, INV  # offsets: with E = 2; gate or dgate alone
        for arg in GOOD[name]:
            if arg in ("dtype", "scale_dtype", "y_dtype"):
                for d in (MOE_FP8_E4M3, 7, -1):
                    yield name, {arg: d}, INV
            if arg in ("T", "n_rows"):
                yield name, {arg: -1}, INV
                yield name, {arg: 8388609}, UNS
            if arg == "T":
                yield name, {arg: 1048577}, UNS
    for kw, want in (({"E": 0}, UNS), ({"E": 257}, UNS), ({"M": 0}, UNS), ({"M": 60}, UNS), ({"M": 65544}, UNS),
                     ({"M": 72, "swiglu": 1}, UNS), ({"swiglu": 2}, INV), ({"swiglu": -1}, INV), ({"K": 0}, UNS),
                     ({"K": -64}, UNS), ({"K": 96}, UNS), ({"K": 16448}, UNS), ({"group": 0}, UNS),
                     ({"group": 16}, UNS), ({"group": 256}, UNS), ({"group": -32}, UNS), ({"group": 128, "K": 64}, UNS)):
        yield "moe_matmul_w4", kw, want
    for name in ("moe_balance_loss", "moe_balance_loss_backward"):
        for kw, want in (({"E": 7}, UNS), ({"E": 257, "R": 257}, UNS), ({"R": 63}, INV), ({"R": 16385}, UNS)):
            yield name, kw, want
    for kw in ({"E": 7}, {"E": 257}, {"E": 0}):
        yield "moe_route_backward", kw, UNS
    # a bf16 element's alignment is enough, less is not
    yield "moe_balance_loss", {"dtype": MOE_BF16, "logits": A + 1}, INV
    yield "moe_balance_loss_backward", {"dtype": MOE_BF16, "dlogits": A + 1}, INV


@pytest.mark.parametrize("name,changed,want", list(bad_calls()),
                         ids=lambda v: v if isinstance(v, str) else str(v))
def test_refused(lib, name, changed, want):
    assert call(lib, name, **changed) == want


@pytest.mark.parametrize("T", [2000, 100000, 1048576])
def test_workspace_refused(lib, T):
    need = lib.moe_balance_workspace_bytes(T, 64)
    assert need > 0
    places = {a: A + (i << 32) for i, a in enumerate(GOOD["moe_balance_loss"]) if a in ALIGN["moe_balance_loss"]}
    for ws, n in ((None, need), (A + (40 << 32), need - 1), (A + (40 << 32) + 2, need), (A + (40 << 32), 0)):
        assert call(lib, "moe_balance_loss", **dict(places, mask=None, T=T, ws=ws, ws_bytes=n)) == MOE_ERR_WORKSPACE
    for arg in places:  # a workspace that another operand lies in
        assert call(lib, "moe_balance_loss", **dict(places, mask=None, T=T, ws=places[arg], ws_bytes=need)) == INV


def test_workspace_sizes(lib):
    for bad in ((-1, 64), (1048577, 64), (4, 0), (4, 257)):
        assert lib.moe_balance_workspace_bytes(*bad) == 0
    assert lib.moe_balance_workspace_bytes(0, 64) == 0


def test_nothing_to_do(lib):
    """No rows or tokens: fine, with nothing enqueued and no pointer needed."""
    for name, count in (("moe_matmul_w4", "n_rows"), ("moe_balance_loss_backward", "T"), ("moe_route_backward", "T")):
        none = {a: None for a in ALIGN[name] if a != "offsets"}
        assert call(lib, name, **{count: 0}, **none) == MOE_OK


def overlaps():
    for name, outs in OUTPUTS.items():
        for out in outs:
            for arg in list(ALIGN[name]) + [a for a in ("mask",) if a in GOOD[name]]:
                if arg != out:
                    yield name, out, arg


@pytest.mark.parametrize("name,out,other", list(overlaps()))
def test_overlap_refused(lib, name, out, other):
    """An output that shares memory with another operand: every operand has a place of its own, 16 MiB
    apart, but for the two."""
    places = {a: A + (i << 24) for i, a in enumerate(GOOD[name]) if a in ALIGN[name] or a == "mask"}
    assert call(lib, name, **dict(places, **{out: places[other]})) == INV


# ----------------------------------------------------------------------------- the binding
T, E, R, N, M, K = 4, 16, 17, 9, 48, 64


def good(device):
    import torch

    def f32(*shape):
        return torch.zeros(shape, device=device)

    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32, device=device)

    def u8(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device=device)

    return {
        "matmul_w4": (binding.matmul_w4, dict(x=f32(N, K), w=u8(2, M, K // 2), scale=f32(2, 2, M), zero=u8(2, 2, M),
                                              offsets=torch.tensor([0, 3, 9], dtype=torch.int32, device=device),
                                              y=f32(N, M))),
        "balance_loss": (binding.balance_loss, dict(logits=f32(T, R), ids=i32(T, 8), num_experts=E,
                                                    mask=u8(T).bool())),
        "balance_loss_backward": (binding.balance_loss_backward,
                                  dict(dloss=f32(), logits=f32(T, R), counts=i32(E), tokens=i32(),
                                       mask=u8(T), dlogits=f32(T, R))),
        "route_backward": (binding.route_backward, dict(dw=f32(T, 8), w=f32(T, 8), ids=i32(T, 8), num_experts=E,
                                                        dgate=f32(T), gate=f32(T), dlogits=f32(T, E + 1))),
    }


def shorter(t):
    return t[1:].contiguous()


def strided(t):
    import torch
    return torch.stack([t, t], dim=-1)[..., 0]


def half(t):
    return t.half()


def long(t):
    return t.long()


def none(t):
    return None


REFUSED = [
    ("matmul_w4", "x", half, "x: dtype"), ("matmul_w4", "x", strided, "x must be contiguous"),
    ("matmul_w4", "x", shorter, "y: shape"), ("matmul_w4", "x", lambda t: t[:, :32].contiguous(), "w: shape"),
    ("matmul_w4", "x", lambda t: t[0], "values to unpack"),
    ("matmul_w4", "w", long, "w: dtype"), ("matmul_w4", "w", strided, "w must be contiguous"),
    ("matmul_w4", "w", shorter, "scale: shape"), ("matmul_w4", "w", lambda t: t[0], "values to unpack"),
    ("matmul_w4", "scale", half, "scale: dtype"), ("matmul_w4", "scale", strided, "scale must be contiguous"),
    ("matmul_w4", "scale", lambda t: t[:, :0], "scale: 0 groups"),
    ("matmul_w4", "scale", lambda t: t.repeat(1, 3, 1), "scale: 6 groups"),
    ("matmul_w4", "scale", lambda t: t[:, :, 8:].contiguous(), "scale: shape"),
    ("matmul_w4", "scale", lambda t: t[:, :1].contiguous(), "zero: shape"),
    ("matmul_w4", "scale", lambda t: t.requires_grad_(), "records no gradient"),
    ("matmul_w4", "x", lambda t: t.requires_grad_(), "records no gradient"),
    ("matmul_w4", "zero", long, "zero: dtype"), ("matmul_w4", "zero", shorter, "zero: shape"),
    ("matmul_w4", "zero", strided, "zero must be contiguous"),
    ("matmul_w4", "offsets", long, "offsets: dtype"), ("matmul_w4", "offsets", shorter, "offsets: shape"),
    ("matmul_w4", "swiglu", lambda _: True, "y: shape"),
    ("matmul_w4", "dtype", lambda _: _bf16(), "y: dtype"),
    ("matmul_w4", "y", half, "y: dtype"), ("matmul_w4", "y", shorter, "y: shape"),
    ("matmul_w4", "y", strided, "y must be contiguous"),
    ("balance_loss", "logits", half, "logits: dtype"), ("balance_loss", "logits", strided, "logits must be contiguous"),
    ("balance_loss", "logits", lambda t: t[:, :16], "logits must be contiguous"),
    ("balance_loss", "logits", lambda t: t[0], "values to unpack"),
    ("balance_loss", "logits", shorter, "ids: shape"),
    ("balance_loss", "ids", long, "ids: dtype"), ("balance_loss", "ids", strided, "ids must be contiguous"),
    ("balance_loss", "ids", shorter, "ids: shape"), ("balance_loss", "ids", lambda t: t[:, :4].contiguous(), "ids: shape"),
    ("balance_loss", "mask", lambda t: t.float(), "mask: dtype"), ("balance_loss", "mask", shorter, "mask: shape"),
    ("balance_loss", "mask", strided, "mask must be contiguous"),
    ("balance_loss_backward", "dloss", lambda t: t.double(), "dloss: dtype"),
    ("balance_loss_backward", "dloss", lambda t: t[None], "dloss: shape"),
    ("balance_loss_backward", "logits", half, "logits: dtype"),
    ("balance_loss_backward", "logits", strided, "logits must be contiguous"),
    ("balance_loss_backward", "logits", shorter, "mask: shape"),
    ("balance_loss_backward", "counts", long, "counts: dtype"),
    ("balance_loss_backward", "counts", lambda t: t[None], "counts: shape"),
    ("balance_loss_backward", "counts", strided, "counts must be contiguous"),
    ("balance_loss_backward", "tokens", long, "tokens: dtype"),
    ("balance_loss_backward", "tokens", lambda t: t[None], "tokens: shape"),
    ("balance_loss_backward", "mask", long, "mask: dtype"), ("balance_loss_backward", "mask", shorter, "mask: shape"),
    ("balance_loss_backward", "dlogits", half, "dlogits: dtype"),
    ("balance_loss_backward", "dlogits", shorter, "dlogits: shape"),
    ("balance_loss_backward", "dlogits", strided, "dlogits must be contiguous"),
    ("route_backward", "dw", half, "dw: dtype"), ("route_backward", "dw", shorter, "dw: shape"),
    ("route_backward", "dw", strided, "dw must be contiguous"),
    ("route_backward", "w", half, "w: dtype"), ("route_backward", "w", shorter, "dw: shape"),
    ("route_backward", "w", strided, "w must be contiguous"),
    ("route_backward", "ids", long, "ids: dtype"), ("route_backward", "ids", strided, "ids must be contiguous"),
    ("route_backward", "dgate", none, "both or neither"), ("route_backward", "gate", none, "both or neither"),
    ("route_backward", "dgate", shorter, "dgate: shape"), ("route_backward", "gate", half, "gate: dtype"),
    ("route_backward", "num_experts", lambda e: e + 1, "dlogits: shape"),
    ("route_backward", "dlogits", half, "dlogits: dtype"), ("route_backward", "dlogits", strided, "dlogits must be"),
]
IDS = [f"{op}-{arg}-{i}" for i, (op, arg, _, _) in enumerate(REFUSED)]
OPERATORS = ("matmul_w4", "balance_loss", "balance_loss_backward", "route_backward")


def _bf16():
    import torch
    return torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """Calls that reach the library, with CPU tensors taken for a device's (number -1 in place of 0)."""
    import torch
    seen = []

    class Library:
        def moe_balance_workspace_bytes(self, tokens, experts):
            return 64

        def __getattr__(self, name):
            return lambda *args: seen.append((name, args)) or binding.MOE_OK

    want = binding._want
    monkeypatch.setattr(binding, "_want", lambda name, t, dtype, shape, at: want(name, t, dtype, shape, -1))
    monkeypatch.setattr(binding, "_switched", lambda device, stream: None)
    monkeypatch.setattr(binding, "load", lambda: Library())
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    return seen


@pytest.mark.parametrize("op", OPERATORS)
def test_good_call_reaches_the_library(calls, op):
    f, operands = good("cpu")[op]
    f(**operands)
    assert [name for name, _ in calls] == ["moe_" + op]
    given = [v.data_ptr() for v in operands.values() if hasattr(v, "data_ptr")]
    assert set(given) <= set(calls[0][1])


@pytest.mark.parametrize("op,arg,change,message", REFUSED, ids=IDS)
def test_binding_refuses(calls, op, arg, change, message):
    f, operands = good("cpu")[op]
    operands[arg] = change(operands.get(arg))
    with pytest.raises(ValueError, match=message):
        f(**operands)
    assert calls == []


@pytest.mark.parametrize("op", OPERATORS)
def test_refused_off_the_gpu(op):
    f, operands = good("cpu")[op]
    with pytest.raises(ValueError, match="tensors must be on a GPU, not on cpu"):
        f(**operands)


def test_balance_loss_records_its_gradient(calls):
    import torch
    f, a = good("cpu")["balance_loss"]
    z = a["logits"].requires_grad_()
    loss, counts, tokens = f(**a)
    assert loss.requires_grad and not counts.requires_grad and not tokens.requires_grad
    loss.backward()
    assert [name for name, _ in calls] == ["moe_balance_loss", "moe_balance_loss_backward"]
    assert calls[1][1][1:5] == (z.data_ptr(), counts.data_ptr(), tokens.data_ptr(), a["mask"].data_ptr())
    assert z.grad.shape == z.shape
    with torch.no_grad():
        assert not f(**a)[0].requires_grad


@pytest.mark.gpu
@pytest.mark.parametrize("op", OPERATORS)
def test_operand_elsewhere_refused(op):
    """Every operand but the one that says where the call runs, left in host memory."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    f, operands = good("cuda")[op]
    where = {"matmul_w4": "x", "balance_loss": "logits", "balance_loss_backward": "logits", "route_backward": "w"}[op]
    for a, v in operands.items():
        if hasattr(v, "cpu") and a != where:
            with pytest.raises(ValueError, match=f"{a} is on cpu, expected cuda:0"):
                f(**dict(operands, **{a: v.cpu()}))
    f(**operands)
