"""SwiGLU of the 8-bit products where the gate is large: every kernel form, gates from -100 to 100 and
at the infinities, against the formula in 64 bits."""
import pytest

from sparse_moe_routing_amd import binding

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -126

# rows, channels, K, experts (0: dense): sizes that the six kernel forms take, dense and by expert
SHAPES = [(4, 272, 144, 0), (1000, 272, 144, 0), (20, 4096, 144, 0), (127, 4096, 144, 0),
          (500, 4096, 512, 0), (4000, 4096, 144, 0), (4, 4096, 144, 3), (4, 272, 144, 3),
          (127, 4096, 144, 3), (127, 1040, 144, 3), (1000, 4096, 512, 3), (4000, 4096, 512, 3)]


def _torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def operands(n, M, K, E, seed):
    """Codes whose sums are single products v c of codes in -127..127, spread over the rows of an
    expert and its gate channels; a gate spans -100..100, an up value goes to 1.6e34."""
    torch = _torch()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    experts, half = max(E, 1), M // 2
    x = torch.zeros((n, K), dtype=torch.int8, device="cuda")
    w = torch.zeros((experts, M, K), dtype=torch.int8, device="cuda")
    x[:, 5] = torch.randint(-127, 128, (n,), generator=g, device="cuda", dtype=torch.int8)
    w[:, :, 5] = torch.randint(-127, 128, (experts, M), generator=g, device="cuda", dtype=torch.int8)
    x[:, K - 1] = 1  # and one more product that is zero in half of the channels
    w[:, ::2, K - 1] = 1
    w_scale = torch.full((experts, M), 100.0 / 127 ** 2, device="cuda")
    w_scale[:, half:] = 1e30
    cuts = torch.linspace(0, n, experts + 1).round().to(torch.int32)
    return x, torch.ones(n, device="cuda"), w, w_scale, cuts


def exact(x, x_scale, w, w_scale, cuts):
    torch = _torch()
    z = torch.cat([(x[a:b].double() @ w[e].double().t().contiguous()) *
                   x_scale[a:b].double()[:, None] * w_scale[e].double()[None, :]
                   for e, (a, b) in enumerate(zip(cuts.tolist(), cuts.tolist()[1:]))])
    return z[:, :z.shape[1] // 2], z[:, z.shape[1] // 2:]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("n,M,K,E", SHAPES)
def test_large_gates(n, M, K, E, out):
    """Three roundings of the gate move silu by at most 3 (1 + |gate|) u; the exponential by halves
    (two steps each), its correction (1), three products (3) and the product with up (3 + 1) add 12 u,
    which the bound's 10 and the 6 u that 3 (1 + |gate|) has over 3 (|gate| - 1) there
    cover. A silu below the normal numbers is off by half of their smallest step."""
    torch = _torch()
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[out]
    x, xs, w, ws, cuts = operands(n, M, K, E, n + M)
    y = binding.matmul_i8(x, xs, w, ws, offsets=cuts.cuda() if E else None, swiglu=True, dtype=dtype)
    gate, up = exact(x, xs, w, ws, cuts)
    want = gate * torch.sigmoid(gate) * up
    rel = (3 * (1 + gate.abs()) + 10) * U + torch.finfo(dtype).eps / 2
    bound = 1.01 * rel * want.abs() + 2.0 ** -149 * up.abs() + TINY
    err = (y.double() - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (int(bad.sum()), gate[bad][:4].tolist(), want[bad][:4].tolist(),
                                 y[bad][:4].tolist())
    if n >= 100:  # the range was met: normal results of gates whose e^-z is past 2^126
        far = (gate < -87.5) & (gate > -91.5) & (up.abs() > 1e32)
        assert bool(far.any()) and bool((y[far] != 0).all())


@pytest.mark.parametrize("n,M,K,E", SHAPES)
def test_infinite_gates(n, M, K, E):
    """A gate of +infinity gives up's sign of it; -infinity and NaN give NaN, as z / (1 + e^-z)."""
    torch = _torch()
    x, xs, w, ws, cuts = operands(n, M, K, E, n + M + 1)
    ws[:, :M // 2:3] = float("inf")
    y = binding.matmul_i8(x, xs, w, ws, offsets=cuts.cuda() if E else None, swiglu=True,
                          dtype=torch.float32)
    gate, up = exact(x, xs, w, ws, cuts)
    want = gate * torch.sigmoid(gate) * up
    infinite = torch.isinf(want)
    assert bool(torch.isnan(want).any()) and bool(infinite.any())
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(y[infinite].double(), want[infinite])
    assert bool(torch.isfinite(y[torch.isfinite(want)]).all())
