"""GPU tests of how exact the products with 4-bit weights are: the number of rows does not decide it.

Rows and a result in bf16 cost one rounding of the result beside what fp32 sums cost, in the forms for few
rows and in those for many. u = 2^-24: a sum of K products takes at most K additions in fp32, each off by at most 2u
(the matrix unit may cut a sum off), and the scale and the zero point's term a few roundings per group, so
that z is off by at most d = (2 K + 8) u sum s |x| (|c - 8| + |z - 8|); with bf16 results by half a step
of the result more. SwiGLU: |silu'| <= 1.1, so that silu(a) b is off by at most 1.1 d_a |b| + |silu(a)| d_b +
1.1 d_a d_b, and 18 u of itself (silu a few fp32 steps, taken as 16, the product one).
"""
import pytest

from sparse_moe_routing_amd import binding
from test_gpu_w4 import U, _torch, dt, gen, plain, split, weights

pytestmark = pytest.mark.gpu

# experts, rows, channels, columns, group: few rows and many
SHAPES = [(1, 4, 1024, 2048, 128), (1, 40, 1024, 1024, 64), (1, 900, 8208, 64, 64), (1, 2700, 2064, 320, 64),
          (1, 5000, 1040, 1152, 128), (1, 1300, 4112, 448, 32), (4, 3300, 2064, 448, 32), (16, 5100, 1552, 192, 32),
          (40, 12000, 2064, 640, 128), (64, 18432, 2064, 192, 64)]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("zero,sdt", [(False, "bf16"), (True, "bf16"), (False, "f32"), (True, "f32")])
@pytest.mark.parametrize("E,n,M,K,G", SHAPES)
def test_bf16_results_are_rounded_once(E, n, M, K, G, zero, sdt, swiglu):
    torch = _torch()
    g = gen(n + K)
    w, scale, z = weights(g, E, M, K, G, zero, sdt, False)
    x = torch.randn((n, K), generator=g, device="cuda").to(torch.bfloat16)
    offsets = None if E == 1 else split(n, E, n)
    want, size, on = plain(x, w, scale, z, offsets)
    y = binding.matmul_w4(x, w, scale, zero=z, offsets=offsets, swiglu=swiglu)
    assert y.dtype is torch.bfloat16
    off = (2 * K + 8) * U * size
    if swiglu:
        h = M // 2
        a, b, da, db = want[:, :h], want[:, h:], off[:, :h], off[:, h:]
        s = a * torch.sigmoid(a)
        want, off = s * b, 1.1 * da * b.abs() + s.abs() * db + 1.1 * da * db
        off = off + 18 * U * want.abs() + 2.0 ** -126
    bad = (y.double() - want).abs() > 1.01 * (off + 2.0 ** -8 * want.abs())
    bad &= on[:, None]
    assert not bool(bad.any()), (int(bad.sum()), bad.numel())


@pytest.mark.parametrize("xdt,ydt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("E,n,M,K,G", SHAPES)
def test_codes_of_their_zero_point_are_nothing(E, n, M, K, G, xdt, ydt):
    """Channels whose codes all equal their group's zero point, under scales of all 24 bits: exactly 0, beside
    channels that are not. Rows are small whole numbers, so that no sum is rounded."""
    torch = _torch()
    g = gen(n + M)
    w, scale, z = weights(g, E, M, K, G, True, "f32", False)
    scale = torch.rand(scale.shape, generator=g, device="cuda") + 0.01
    same = z | (z << 4)  # both codes of a byte
    none = torch.arange(M, device="cuda") % 3 == 1
    spread = same.transpose(1, 2).repeat_interleave(G // 2, dim=2)
    w = torch.where(none[None, :, None], spread, w)
    x = torch.randint(-3, 4, (n, K), generator=g, device="cuda").to(dt(xdt))
    offsets = None if E == 1 else split(n, E, n)
    y = torch.zeros((n, M), dtype=dt(ydt), device="cuda")
    binding.matmul_w4(x, w, scale, zero=z, offsets=offsets, y=y)
    assert bool((y[:, none] == 0).all()), int((y[:, none] != 0).sum())
    assert bool((y[:, ~none] != 0).any())
