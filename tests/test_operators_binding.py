"""The binding's checks of the separate operators, argument by argument: a good call with one operand
changed raises ValueError with the message of that check, and the library is not called. The
same table runs on the CPU, with the library and the device lookup stood in for, and on the GPU
as users call it."""
import pytest

from sparse_moe_routing_amd import binding

T, H, N, E, M, K = 4, 64, 32, 2, 48, 64


def good(device):
    """(function, its good operands) of every operator."""
    import torch

    def f32(*shape):
        return torch.zeros(shape, device=device)

    def i8(*shape):
        return torch.zeros(shape, dtype=torch.int8, device=device)

    def rows():
        return torch.arange(N, dtype=torch.int32, device=device)

    def offsets():
        return torch.tensor([0, 3, 9], dtype=torch.int32, device=device)

    return {
        "permute": (binding.permute, dict(x=f32(T, H), rows=rows(), n_rows=N, xs=f32(N, H))),
        "permute_backward": (binding.permute_backward, dict(dxs=f32(N, H), rows=rows(),
                                                            dx=f32(T, H))),
        "unpermute": (binding.unpermute, dict(ys=f32(N, H), rows=rows(), w=f32(T, 8),
                                              shared=f32(T, H), gate=f32(T), y=f32(T, H))),
        "unpermute_backward": (binding.unpermute_backward,
                               dict(dy=f32(T, H), ys=f32(N, H), rows=rows(), w=f32(T, 8),
                                    shared=f32(T, H), gate=f32(T), dys=f32(N, H))),
        "quantize_i8": (binding.quantize_i8, dict(x=f32(T, H))),
        "permute_i8": (binding.permute_i8, dict(x=f32(T, H), rows=rows(), n_rows=N)),
        "matmul_i8": (binding.matmul_i8, dict(x=i8(9, K), x_scale=f32(9), w=i8(E, M, K),
                                              w_scale=f32(E, M), offsets=offsets(), y=f32(9, M))),
    }


def shorter(t):
    return t[1:].contiguous()


def narrower(t):
    return t[..., 8:].contiguous()


def strided(t):
    import torch
    return torch.stack([t, t], dim=-1)[..., 0]


def half(t):
    return t.half()


def long(t):
    return t.long()


def double(t):
    return t.double()


def none(t):
    return None


# operator, operand, change, the check's message
REFUSED = [
    ("permute", "x", half, "x: dtype"), ("permute", "x", strided, "x must be contiguous"),
    ("permute", "x", lambda t: t[None], "values to unpack"),
    ("permute", "x", shorter, "rows: shape"), ("permute", "x", narrower, "xs: shape"),
    ("permute", "rows", long, "rows: dtype"), ("permute", "rows", shorter, "rows: shape"),
    ("permute", "rows", lambda t: t.reshape(T, 8), "rows: shape"),
    ("permute", "rows", strided, "rows must be contiguous"),
    ("permute", "n_rows", lambda n: n + 1, "xs: shape"),
    ("permute", "xs", half, "xs: dtype"), ("permute", "xs", shorter, "xs: shape"),
    ("permute", "xs", narrower, "xs: shape"), ("permute", "xs", strided, "xs must be contiguous"),
    ("permute_backward", "dxs", half, "dxs: dtype"),
    ("permute_backward", "dxs", strided, "dxs must be contiguous"),
    ("permute_backward", "dxs", narrower, "dx: shape"),
    ("permute_backward", "rows", long, "rows: dtype"),
    ("permute_backward", "rows", shorter, "rows: shape"),
    ("permute_backward", "dx", half, "dx: dtype"), ("permute_backward", "dx", shorter, "dx: shape"),
    ("permute_backward", "dx", strided, "dx must be contiguous"),
    ("unpermute", "ys", half, "ys: dtype"), ("unpermute", "ys", strided, "ys must be contiguous"),
    ("unpermute", "ys", narrower, "shared: shape"),
    ("unpermute", "rows", long, "rows: dtype"), ("unpermute", "rows", shorter, "rows: shape"),
    ("unpermute", "w", double, "w: dtype"), ("unpermute", "w", shorter, "rows: shape"),
    ("unpermute", "w", lambda t: t[:, :7].contiguous(), "w: shape"),
    ("unpermute", "w", strided, "w must be contiguous"),
    ("unpermute", "shared", none, "both or neither"), ("unpermute", "gate", none, "both or neither"),
    ("unpermute", "shared", half, "shared: dtype"), ("unpermute", "shared", shorter, "shared: shape"),
    ("unpermute", "shared", strided, "shared must be contiguous"),
    ("unpermute", "gate", double, "gate: dtype"), ("unpermute", "gate", shorter, "gate: shape"),
    ("unpermute", "gate", strided, "gate must be contiguous"),
    ("unpermute", "dtype", lambda _: binding_dtype("bfloat16"), "y: dtype"),
    ("unpermute", "y", half, "y: dtype"), ("unpermute", "y", shorter, "y: shape"),
    ("unpermute", "y", strided, "y must be contiguous"),
    ("unpermute_backward", "dy", half, "dy: dtype"),
    ("unpermute_backward", "dy", shorter, "dy: shape"),
    ("unpermute_backward", "dy", narrower, "dy: shape"),
    ("unpermute_backward", "dy", strided, "dy must be contiguous"),
    ("unpermute_backward", "ys", half, "ys: dtype"),
    ("unpermute_backward", "ys", narrower, "dy: shape"),
    ("unpermute_backward", "ys", strided, "ys must be contiguous"),
    ("unpermute_backward", "rows", long, "rows: dtype"),
    ("unpermute_backward", "rows", shorter, "rows: shape"),
    ("unpermute_backward", "w", double, "w: dtype"),
    ("unpermute_backward", "w", shorter, "dy: shape"),
    ("unpermute_backward", "shared", none, "both or neither"),
    ("unpermute_backward", "gate", none, "both or neither"),
    ("unpermute_backward", "shared", shorter, "shared: shape"),
    ("unpermute_backward", "gate", shorter, "gate: shape"),
    ("unpermute_backward", "dys", half, "dys: dtype"),
    ("unpermute_backward", "dys", shorter, "dys: shape"),
    ("unpermute_backward", "dys", strided, "dys must be contiguous"),
    ("quantize_i8", "x", half, "x: dtype"), ("quantize_i8", "x", strided, "x must be contiguous"),
    ("quantize_i8", "x", lambda t: t[0], "values to unpack"),
    ("permute_i8", "x", half, "x: dtype"), ("permute_i8", "x", strided, "x must be contiguous"),
    ("permute_i8", "x", shorter, "rows: shape"), ("permute_i8", "rows", long, "rows: dtype"),
    ("permute_i8", "rows", shorter, "rows: shape"),
    ("matmul_i8", "x", long, "x: dtype"), ("matmul_i8", "x", strided, "x must be contiguous"),
    ("matmul_i8", "x", narrower, "w: shape"), ("matmul_i8", "x", shorter, "x_scale: shape"),
    ("matmul_i8", "x_scale", double, "x_scale: dtype"),
    ("matmul_i8", "x_scale", shorter, "x_scale: shape"),
    ("matmul_i8", "x_scale", strided, "x_scale must be contiguous"),
    ("matmul_i8", "w", long, "w: dtype"), ("matmul_i8", "w", strided, "w must be contiguous"),
    ("matmul_i8", "w", lambda t: t[0], "values to unpack"),
    ("matmul_i8", "w", shorter, "w_scale: shape"),
    ("matmul_i8", "w_scale", double, "w_scale: dtype"),
    ("matmul_i8", "w_scale", narrower, "w_scale: shape"),
    ("matmul_i8", "w_scale", shorter, "w_scale: shape"),
    ("matmul_i8", "w_scale", strided, "w_scale must be contiguous"),
    ("matmul_i8", "offsets", long, "offsets: dtype"),
    ("matmul_i8", "offsets", shorter, "offsets: shape"),
    ("matmul_i8", "offsets", strided, "offsets must be contiguous"),
    ("matmul_i8", "swiglu", lambda _: True, "y: shape"),
    ("matmul_i8", "dtype", lambda _: binding_dtype("bfloat16"), "y: dtype"),
    ("matmul_i8", "y", half, "y: dtype"), ("matmul_i8", "y", shorter, "y: shape"),
    ("matmul_i8", "y", narrower, "y: shape"), ("matmul_i8", "y", strided, "y must be contiguous"),
]
IDS = [f"{op}-{arg}-{i}" for i, (op, arg, _, _) in enumerate(REFUSED)]
OPERATORS = ("permute", "permute_backward", "unpermute", "unpermute_backward", "quantize_i8",
             "permute_i8", "matmul_i8")


def binding_dtype(name):
    import torch
    return getattr(torch, name)


def refuse(device, op, arg, change, message):
    f, operands = good(device)[op]
    operands[arg] = change(operands.get(arg))
    with pytest.raises(ValueError, match=message):
        f(**operands)


@pytest.fixture
def calls(monkeypatch):
    """Calls that reach the library, as [(entry point, arguments)], with CPU tensors taken for a
    device's: their device number is -1 where a GPU's is its index."""
    import torch
    seen = []

    class Library:
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
    """What the refusals change is all that is wrong with them; addresses go in as given."""
    f, operands = good("cpu")[op]
    f(**operands)
    assert [name for name, _ in calls] == ["moe_" + op]
    given = [v.data_ptr() for v in operands.values() if hasattr(v, "data_ptr")]
    assert set(given) <= set(calls[0][1])


@pytest.mark.parametrize("op,arg,change,message", REFUSED, ids=IDS)
def test_refused(calls, op, arg, change, message):
    refuse("cpu", op, arg, change, message)
    assert calls == []


@pytest.mark.parametrize("op", OPERATORS)
def test_refused_off_the_gpu(op):
    f, operands = good("cpu")[op]
    with pytest.raises(ValueError, match="tensors must be on a GPU, not on cpu"):
        f(**operands)


def needs_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


@pytest.mark.gpu
@pytest.mark.parametrize("op,arg,change,message", REFUSED, ids=IDS)
def test_refused_on_the_gpu(op, arg, change, message):
    needs_gpu()
    refuse("cuda", op, arg, change, message)


@pytest.mark.gpu
@pytest.mark.parametrize("op", OPERATORS)
def test_operand_elsewhere_refused(op):
    """Every operand but the first, which says where the call runs, left in host memory."""
    needs_gpu()
    f, operands = good("cuda")[op]
    names = [a for a, v in operands.items() if hasattr(v, "cpu")]
    first = "ys" if "ys" in names else names[0]
    for a in names:
        if a != first:
            with pytest.raises(ValueError, match=f"{a} is on cpu, expected cuda:0"):
                f(**dict(operands, **{a: operands[a].cpu()}))
    f(**operands)


@pytest.mark.gpu
def test_misaligned_rows_refused():
    """Contiguous views that begin off a 16-byte boundary are the library's to refuse."""
    torch = needs_gpu()
    room = torch.zeros(N * H + 1, device="cuda")
    for op, arg, shape in (("permute", "x", (T, H)), ("permute", "xs", (N, H)),
                           ("unpermute", "ys", (N, H)), ("quantize_i8", "x", (T, H))):
        f, operands = good("cuda")[op]
        operands[arg] = room[1:1 + shape[0] * shape[1]].view(shape)
        with pytest.raises(binding.MoeError) as e:
            f(**operands)
        assert e.value.status == binding.MOE_ERR_INVALID_ARG


# ----------------------------------------------------------------------------- autograd
def test_permute_records_its_gradient(calls):
    """A tensor that requires a gradient gets it through the library's gradient operator, on a
    contiguous, 16-byte aligned copy where autograd's own is neither."""
    import torch
    f, a = good("cpu")["permute"]
    x = a["x"].requires_grad_()
    xs = f(x, a["rows"])
    assert xs.requires_grad and [name for name, _ in calls] == ["moe_permute"]
    xs.sum().backward()  # an expanded gradient
    assert [name for name, _ in calls] == ["moe_permute", "moe_permute_backward"]
    address, rows = calls[1][1][:2]
    assert rows == a["rows"].data_ptr() and address % 16 == 0
    assert x.grad.shape == x.shape
    room = torch.zeros(N * H + 1)
    f(x, a["rows"]).backward(room[1:].view(N, H))  # a view off the boundary
    assert calls[3][1][0] % 16 == 0


@pytest.mark.parametrize("arg", ["ys", "w", "shared", "gate"])
def test_unpermute_records_its_gradients(calls, arg):
    f, a = good("cpu")["unpermute"]
    del a["y"]
    a[arg].requires_grad_()
    y = f(**a)
    assert y.requires_grad and [name for name, _ in calls] == ["moe_unpermute"]
    y.sum().backward()
    assert [name for name, _ in calls] == ["moe_unpermute", "moe_unpermute_backward"]
    assert calls[1][1][1:6] == tuple(a[k].data_ptr() for k in ("ys", "rows", "w", "shared", "gate"))
    for k in ("ys", "w", "shared", "gate"):
        assert (a[k].grad is not None) == (k == arg)


def test_buffers_and_gradients_exclude_each_other(calls):
    """A result buffer while a gradient is recorded is refused; without recording it is filled."""
    import torch
    for op, arg, out in (("permute", "x", "xs"), ("unpermute", "ys", "y"), ("unpermute", "w", "y"),
                         ("unpermute", "shared", "y"), ("unpermute", "gate", "y")):
        f, a = good("cpu")[op]
        a[arg].requires_grad_()
        with pytest.raises(ValueError, match=f"{out} cannot be given where a gradient is recorded"):
            f(**a)
        assert calls == []
        with torch.no_grad():
            assert f(**a) is a[out] and not a[out].requires_grad
            del a[out]
            assert not f(**a).requires_grad
        assert [name for name, _ in calls] == ["moe_" + op] * 2
        calls.clear()


def test_refusals_hold_where_a_gradient_is_recorded(calls):
    import torch
    f, a = good("cpu")["permute"]
    with pytest.raises(ValueError, match="rows: dtype"):
        f(a["x"].requires_grad_(), a["rows"].long())
    f, a = good("cpu")["unpermute"]
    with pytest.raises(ValueError, match="both or neither"):
        f(a["ys"], a["rows"], a["w"].requires_grad_(), gate=a["gate"])
    assert calls == []
    # a second derivative is refused, not dropped
    f, a = good("cpu")["permute"]
    x = a["x"].requires_grad_()
    dx, = torch.autograd.grad(f(x, a["rows"]).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()


# ----------------------------------------------------------------------------- the layer's calls
@pytest.fixture
def layer(monkeypatch):
    """A MoeLayer without a device: its library answers every call with success and writes (entry
    point, arguments) down, next to the stream that each zeroed allocation was made on."""
    import contextlib

    import torch
    m = binding.MoeLayer.__new__(binding.MoeLayer)
    m.ctx, m.num_experts, m.shared_inter, m.rows, m.hidden = None, 16, 0, 16, 64
    m.seen, now = [], [None]

    class Library:
        def moe_workspace_bytes(self, ctx, tokens):
            return 512

        def __getattr__(self, name):
            return lambda *args: m.seen.append((name, args)) or binding.MOE_OK

    m.lib = Library()
    zeros = torch.zeros

    @contextlib.contextmanager
    def on(stream):
        before, now[0] = now[0], stream if stream is not None else now[0]
        yield
        now[0] = before

    def noted(*args, **kwargs):
        m.seen.append(("zeros", now[0]))
        return zeros(*args, **kwargs)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "zeros", noted)
    monkeypatch.setattr(binding, "_stream", lambda stream=None: now[0] if stream is None else stream)
    monkeypatch.setattr(binding, "_switched", lambda device, stream: None if stream is None else on(stream))
    want = binding._want
    monkeypatch.setattr(binding, "_want", lambda name, t, dtype, shape, at: want(name, t, dtype, shape, -1))
    return m


LAYER_CALLS = {
    "route": lambda m, x, ids, **k: m.route(x=x, **k),
    "bucket": lambda m, x, ids, **k: m.bucket(ids, **k),
    "bucket_rows": lambda m, x, ids, **k: m.bucket_rows(ids, **k),
    "forward": lambda m, x, ids, **k: m.forward(x, **k),
}


@pytest.mark.parametrize("name", list(LAYER_CALLS))
def test_workspace_is_zeroed_on_the_calls_stream(layer, name):
    """Without a workspace of the caller's the call zeroes one: on the stream that its kernels are
    enqueued on, or nothing orders the fill before them."""
    import torch
    x, ids = torch.ones(4, 64), torch.ones((4, 8), dtype=torch.int32)
    for stream in (None, "side"):
        layer.seen.clear()
        LAYER_CALLS[name](layer, x, ids, stream=stream)
        assert layer.seen[0] == ("zeros", stream)
        assert layer.seen[1][0] == "moe_" + name and stream in layer.seen[1][1]
        assert len(layer.seen) == 2


BAD_IDS = [(long, "ids: dtype"), (lambda t: t.float(), "ids: dtype"), (strided, "ids must be contiguous"),
           (lambda t: t.reshape(-1), "ids: shape"), (lambda t: t[:, :4].contiguous(), "ids: shape"),
           (lambda t: t.t(), "ids: shape")]


@pytest.mark.parametrize("change,message", BAD_IDS, ids=[str(i) for i in range(len(BAD_IDS))])
def test_bucket_rows_refuses_ids(layer, change, message):
    """ids of another type or layout would be read as other experts' numbers."""
    import torch
    with pytest.raises(ValueError, match=message):
        layer.bucket_rows(change(torch.ones((4, 8), dtype=torch.int32)))
    assert layer.seen == []


def test_bucket_rows_refuses_host_ids():
    import torch
    m = binding.MoeLayer.__new__(binding.MoeLayer)
    with pytest.raises(ValueError, match="tensors must be on a GPU, not on cpu"):
        m.bucket_rows(torch.ones((4, 8), dtype=torch.int32))


@pytest.mark.gpu
def test_bucket_rows_refuses_on_the_gpu():
    torch = needs_gpu()
    from sparse_moe_routing_amd import inputs
    m, t = binding.layer_from_numpy(inputs.make_layer(inputs.BY_NAME["tiny_fp32_t4"]), 64)
    ids = m.route(x=t["x"])[1]
    for change, message in BAD_IDS:
        with pytest.raises(ValueError, match=message):
            m.bucket_rows(change(ids))
    assert torch.equal(m.bucket_rows(ids)[2], m.bucket(ids)[2])
    m.close()


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(LAYER_CALLS))
def test_layer_call_on_a_side_stream(name):
    """The same results on a side stream while the current one is busy and its freed memory holds
    other values."""
    torch = needs_gpu()
    from sparse_moe_routing_amd import inputs
    m, t = binding.layer_from_numpy(inputs.make_layer(inputs.BY_NAME["tiny_fp32_t4"]), 64)
    ids = m.route(x=t["x"])[1]

    def results(stream=None):
        out = LAYER_CALLS[name](m, t["x"], ids, stream=stream)
        return [v for v in (out if isinstance(out, tuple) else (out,)) if v is not None]

    want = results()
    side = torch.cuda.Stream()
    busy = torch.ones(1 << 26, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        # what the current stream's allocator hands out next holds ones
        torch.full((m.workspace_bytes(64),), 1, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for _ in range(8):
            busy.mul_(1.0)
        got = results(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    m.close()
