"""GPU tests of the products with 4-bit weights against plain 64-bit forms.

Whole numbers: rows and zeros are whole numbers and scales powers of two, so small that every sum is a
multiple of one power of two below 2^24 of them: fp32 holds every partial sum exactly in any order, and
fp32 results are compared for equality, bf16 ones with the one rounding of the exact sum.

Drawn numbers: u = 2^-24. A sum of K products takes at most K additions in fp32; the matrix unit may cut
a sum off instead of rounding it, which is up to 2u. The scale and the zero point's term cost a few more
roundings per group. So the error is at most (2 K + 8) u times the sum of the terms' absolute values
s |x| (|c - 8| + |z - 8|), and half a step of the result's type.
With bf16 rows and a bf16 result a product of many rows rounds its weights s (c - z) to bf16, as documented:
each by at most h = 2^-8 of itself, so that the sum moves by at most h sum |x| |s (c - z)|, which is at most h
times the same sum of absolute values (|c - z| <= |c - 8| + |z - 8|).
"""
import pytest

from sparse_moe_routing_amd import binding

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def dt(name):
    torch = _torch()
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def gen(seed):
    torch = _torch()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def weights(g, E, M, K, G, zero, sdt, whole):
    torch = _torch()
    w = torch.randint(0, 256, (E, M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    shape = (E, K // G, M)
    if whole:
        scale = 2.0 ** torch.randint(-3, 1, shape, generator=g, device="cuda").float()
    else:
        scale = torch.rand(shape, generator=g, device="cuda") * 0.01 + 1e-3
    z = torch.randint(0, 16, shape, generator=g, device="cuda").to(torch.uint8) if zero else None
    return w, scale.to(dt(sdt)), z


def spread(w, scale, z, e):
    """(codes, zeros, scales) of expert e as fp64 [M][K]."""
    torch = _torch()
    M, half = w.shape[1:]
    G = 2 * half // scale.shape[1]
    c = torch.empty((M, 2 * half), dtype=torch.float64, device="cuda")
    c[:, 0::2], c[:, 1::2] = (w[e] & 15).double(), (w[e] >> 4).double()
    s = scale[e].double().t().repeat_interleave(G, dim=1)
    zz = torch.full_like(s, 8.0) if z is None else z[e].double().t().repeat_interleave(G, dim=1)
    return c, zz, s


def plain(x, w, scale, z, offsets):
    """(products, sums of the terms' absolute values) in 64 bits, and which rows have an expert."""
    torch = _torch()
    n, M = x.shape[0], w.shape[1]
    y = torch.zeros((n, M), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(y)
    on = torch.zeros((n,), dtype=torch.bool, device="cuda")
    at = [0, n] if offsets is None else offsets.tolist()
    for e in range(w.shape[0]):
        a, b = min(max(at[e], 0), n), min(max(at[e + 1], 0), n)
        if a >= b:
            continue
        c, zz, s = spread(w, scale, z, e)
        xe = x[a:b].double()
        y[a:b] = xe @ ((c - zz) * s).t().contiguous()
        size[a:b] = xe.abs() @ (((c - 8).abs() + (zz - 8).abs()) * s).t().contiguous()
        on[a:b] = True
    return y, size, on


def swiglu_of(z):
    torch = _torch()
    h = z.shape[1] // 2
    return z[:, :h] * torch.sigmoid(z[:, :h]) * z[:, h:]


def split(n, E, seed, before=0, after=0, hot=False):
    """offsets [E + 1] of n rows, `before` rows of no expert in front and `after` behind; some experts
    have none, and with `hot` one has most."""
    torch = _torch()
    g = torch.Generator()
    g.manual_seed(seed)
    left = n - before - after
    p = torch.rand((E,), generator=g) * (torch.rand((E,), generator=g) < 0.7)
    if hot or float(p.sum()) == 0:
        p[E // 2] = 3.0 * E
    counts = torch.multinomial(p, left, replacement=True, generator=g) if left else torch.zeros(0)
    counts = torch.bincount(counts.long(), minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[0] = before
    off[1:] = before + counts.cumsum(0)
    return off.cuda()


def run_whole(n, E, M, K, G, zero, sdt, xdt, ydt, swiglu, seed, dense=False, before=0, after=0,
              hot=False):
    torch = _torch()
    g = gen(seed)
    w, scale, z = weights(g, E, M, K, G, zero, sdt, True)
    # |sum| <= K 16 xmax below 2^24 eighths
    xmax = max(1, min(9, 2 ** 21 // (K * 16) - 1))
    x = torch.randint(-xmax, xmax + 1, (n, K), generator=g, device="cuda").to(dt(xdt))
    offsets = None if dense else split(n, E, seed, before, after, hot)
    Mo = M // 2 if swiglu else M
    y = torch.full((n, Mo), 7.5, dtype=dt(ydt), device="cuda")
    got = binding.matmul_w4(x, w, scale, zero=z, offsets=offsets, swiglu=swiglu, y=y)
    assert got is y
    want, _, on = plain(x, w, scale, z, offsets)
    if swiglu:
        want = swiglu_of(want)
        half = torch.finfo(y.dtype).eps / 2 if ydt == "bf16" else 0.0
        # silu: a few fp32 steps (taken as 16), the product one
        bad = (y.double() - want).abs() > want.abs() * (half * 1.01 + 18 * U) + 2.0 ** -126
        bad &= on[:, None]
        bad |= ~on[:, None] & (y.double() != 7.5)
        assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())
        return
    want = torch.where(on[:, None], want.float().to(y.dtype), torch.full_like(y, 7.5))
    bad = y != want
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist(),
                                 y[bad][:4].tolist(), want[bad][:4].tolist())


# rows, channels, columns, group: one row and one group, channels that end inside a tile, columns that are
# an odd number of groups, and rows around every tile's edge
DENSE = [(1, 8, 32, 32), (1, 24, 96, 32), (2, 1032, 128, 128), (3, 40, 320, 64), (4, 1024, 2048, 128),
         (5, 72, 1056, 32), (8, 264, 640, 128), (9, 136, 192, 64), (16, 4096, 512, 128), (17, 520, 1024, 64),
         (31, 200, 480, 32), (33, 1000, 256, 128), (48, 88, 2176, 128), (64, 2048, 1024, 128),
         (65, 256, 96, 32), (127, 392, 704, 64), (129, 1288, 384, 128), (256, 512, 512, 32),
         (320, 264, 1152, 128), (321, 248, 160, 32), (700, 1032, 288, 32), (1500, 2056, 640, 128)]


@pytest.mark.parametrize("xdt,ydt,sdt,zero", [("bf16", "bf16", "bf16", False), ("bf16", "f32", "f32", True),
                                              ("f32", "f32", "bf16", True), ("f32", "f32", "f32", False),
                                              ("bf16", "f32", "bf16", False)])
@pytest.mark.parametrize("n,M,K,G", DENSE)
def test_dense_whole_numbers(n, M, K, G, xdt, ydt, sdt, zero):
    run_whole(n, 1, M, K, G, zero, sdt, xdt, ydt, False, 100 + n, dense=True)


@pytest.mark.parametrize("xdt,ydt,zero", [("bf16", "bf16", False), ("f32", "f32", True), ("bf16", "f32", True)])
@pytest.mark.parametrize("n,M,K,G", [(1, 16, 32, 32), (4, 1024, 2048, 128), (7, 48, 96, 32), (19, 208, 640, 128),
                                     (50, 1040, 192, 64), (130, 528, 1152, 128), (400, 272, 352, 32)])
def test_dense_swiglu(n, M, K, G, xdt, ydt, zero):
    run_whole(n, 1, M, K, G, zero, "bf16", xdt, ydt, True, 200 + n, dense=True)


# experts, rows, channels, columns, group
GROUPED = [(8, 3, 24, 64, 32), (256, 32, 64, 256, 128), (60, 61, 136, 96, 32), (16, 200, 1032, 320, 64),
           (255, 256, 512, 512, 128), (64, 700, 264, 704, 64), (8, 1000, 256, 640, 128), (256, 1536, 128, 160, 32),
           (5, 1700, 520, 1024, 128), (256, 9000, 48, 288, 32), (128, 5000, 256, 1280, 128)]


@pytest.mark.parametrize("hot", [False, True])
@pytest.mark.parametrize("xdt,ydt,sdt,zero", [("bf16", "bf16", "bf16", False), ("bf16", "f32", "f32", True),
                                              ("f32", "f32", "bf16", False), ("f32", "bf16", "bf16", True)])
@pytest.mark.parametrize("E,n,M,K,G", GROUPED)
def test_grouped_whole_numbers(E, n, M, K, G, xdt, ydt, sdt, zero, hot):
    run_whole(n, E, M, K, G, zero, sdt, xdt, ydt, False, 300 + n, before=n // 9, after=n // 7, hot=hot)


# few rows and channels, many columns: K split among the waves of a block, in shares that do not come out even
@pytest.mark.parametrize("xdt,ydt,sdt,zero", [("bf16", "bf16", "bf16", False), ("bf16", "f32", "f32", True),
                                              ("f32", "f32", "bf16", False), ("f32", "f32", "bf16", True)])
@pytest.mark.parametrize("n,M,K,G", [(2, 272, 4224, 128), (4, 64, 16384, 64), (7, 272, 2336, 32), (8, 528, 4096, 128),
                                     (14, 144, 4224, 64), (16, 256, 8192, 128), (30, 272, 4096, 32),
                                     (8, 6400, 4224, 64), (15, 6416, 2336, 32)])
def test_split_columns_whole_numbers(n, M, K, G, xdt, ydt, sdt, zero):
    run_whole(n, 1, M, K, G, zero, sdt, xdt, ydt, False, 900 + n, dense=True)
    run_whole(n, 1, M, K, G, zero, sdt, xdt, ydt, True, 950 + n, dense=True)


# many rows an expert: blocks of every height, rows that end inside a block's subtiles, with zero points and
# both scale types on bf16 results (their scales are rounded into the weights, which are exact here)
MANY = [(1, 2700, 2056, 320, 64), (1, 5000, 1032, 1152, 128), (1, 1300, 4104, 448, 32), (1, 900, 8208, 64, 64),
        (4, 3300, 2064, 448, 32), (3, 2950, 2056, 256, 128), (40, 9000, 1032, 704, 64), (16, 5100, 1544, 192, 32),
        (2, 700, 8200, 640, 64), (12, 2000, 4104, 128, 128)]


@pytest.mark.parametrize("xdt,ydt,sdt,zero", [("bf16", "bf16", "bf16", False), ("bf16", "bf16", "f32", True),
                                              ("bf16", "bf16", "bf16", True), ("bf16", "bf16", "f32", False),
                                              ("bf16", "f32", "bf16", False), ("bf16", "f32", "bf16", True),
                                              ("f32", "f32", "bf16", False), ("f32", "f32", "f32", True)])
@pytest.mark.parametrize("E,n,M,K,G", MANY)
def test_many_rows_whole_numbers(E, n, M, K, G, xdt, ydt, sdt, zero):
    run_whole(n, E, M, K, G, zero, sdt, xdt, ydt, False, 700 + n, dense=E == 1, before=0 if E == 1 else 3,
              after=0 if E == 1 else 5)
    run_whole(n, E, M // 16 * 16, K, G, zero, sdt, xdt, ydt, True, 800 + n, dense=E == 1)


@pytest.mark.parametrize("hot", [False, True])
@pytest.mark.parametrize("E,n,M,K,G", GROUPED)
def test_grouped_swiglu(E, n, M, K, G, hot):
    if M % 16:
        M += 8
    run_whole(n, E, M, K, G, False, "bf16", "bf16", "bf16", True, 400 + n, after=n // 5, hot=hot)
    run_whole(n, E, M, K, G, True, "f32", "f32", "f32", True, 500 + n, hot=hot)
    run_whole(n, E, M, K, G, False, "bf16", "f32", "bf16", True, 1000 + n, hot=hot)
    run_whole(n, E, M, K, G, True, "bf16", "bf16", "bf16", True, 1100 + n, hot=hot)


@pytest.mark.parametrize("xdt", ["bf16", "f32"])
@pytest.mark.parametrize("E,n,M,K,G,zero", [(1, 1, 512, 16384, 128, False), (1, 12, 264, 4096, 32, True),
                                            (1, 300, 520, 4096, 64, True), (1, 2100, 1024, 2048, 128, False),
                                            (16, 40, 256, 2048, 128, True), (64, 3000, 256, 1024, 64, False)])
def test_drawn_numbers(E, n, M, K, G, zero, xdt):
    torch = _torch()
    g = gen(600 + n)
    w, scale, z = weights(g, E, M, K, G, zero, "f32", False)
    x = torch.randn((n, K), generator=g, device="cuda").to(dt(xdt))
    offsets = None if E == 1 else split(n, E, n)
    want, size, _ = plain(x, w, scale, z, offsets)
    for out in (torch.float32, torch.bfloat16):
        y = binding.matmul_w4(x, w, scale, zero=z, offsets=offsets, dtype=out)
        half = torch.finfo(out).eps / 2
        rounded = half * size if xdt == "bf16" and out is torch.bfloat16 else 0.0
        bad = (y.double() - want).abs() > 1.01 * ((2 * K + 8) * U * size + rounded + half * want.abs())
        assert not bool(bad.any()), (out, int(bad.sum()))
    # far inside the bound on the whole: fp32 results as near as an fp32 product of the same size gets
    y = binding.matmul_w4(x, w, scale, zero=z, offsets=offsets, dtype=torch.float32)
    rel = float((y.double() - want).norm() / want.norm())
    assert rel < 2e-6, rel


def test_all_of_fp32_counts():
    """Rows whose elements use all 24 bits, against one channel of weight 1: the row's sum is exact."""
    torch = _torch()
    g = gen(7)
    for n in (1, 5, 40, 200):
        x = torch.zeros((n, 64), device="cuda")
        at = torch.randint(0, 64, (n,), generator=g, device="cuda")
        v = 1.0 + torch.randint(0, 2 ** 23, (n,), generator=g, device="cuda").double() / 2 ** 23
        x[torch.arange(n), at] = v.float()
        w = torch.full((1, 8, 32), 0x99, dtype=torch.uint8, device="cuda")  # 9 - 8 = 1
        y = binding.matmul_w4(x, w, torch.ones((1, 2, 8), device="cuda"), dtype=torch.float32)
        assert torch.equal(y, v.float()[:, None].expand(n, 8))


def test_every_code_and_zero():
    """One column at a time: code - zero of all 16 codes and of zeros from 0 to 255."""
    torch = _torch()
    K = 32
    x = torch.eye(K, device="cuda").to(torch.bfloat16)
    zeros = torch.arange(256, dtype=torch.uint8, device="cuda").reshape(1, 1, 256).contiguous()
    w = torch.empty((1, 256, K // 2), dtype=torch.uint8, device="cuda")
    w[:] = (torch.arange(16, device="cuda") | (torch.arange(16, device="cuda").flip(0) << 4)).to(torch.uint8)
    code = torch.stack([torch.arange(16), torch.arange(16).flip(0)], 1).reshape(-1).cuda().float()
    one = torch.ones((1, 1, 256), device="cuda")
    y = binding.matmul_w4(x, w, one, zero=zeros, dtype=torch.float32)
    assert torch.equal(y, code[:, None] - torch.arange(256, device="cuda").float()[None, :])
    y = binding.matmul_w4(x, w, one, dtype=torch.float32)
    assert torch.equal(y, (code - 8)[:, None].expand(K, 256))


@pytest.mark.parametrize("xdt", ["bf16", "f32"])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("n", [3, 16, 90, 400])
def test_infinities_stay_in_their_row(n, zero, xdt):
    torch = _torch()
    g = gen(n)
    w, scale, z = weights(g, 1, 72, 192, 64, zero, "bf16", True)
    x = torch.randint(-4, 5, (n, 192), generator=g, device="cuda").to(dt(xdt))
    clean = binding.matmul_w4(x, w, scale, zero=z, dtype=torch.float32)
    x[1, 5], x[n - 1, 191] = float("inf"), float("nan")
    y = binding.matmul_w4(x, w, scale, zero=z, dtype=torch.float32)
    rest = [i for i in range(n) if i not in (1, n - 1)]
    assert torch.equal(y[rest], clean[rest])
    assert bool(y[n - 1].isnan().all())
    assert not bool(y[1].isfinite().any()) or not zero  # inf * 0 is a NaN, inf * c an infinity
    assert not bool(y[1][(w[0, :, 2] >> 4) != 8].isfinite().any())


def test_gates_far_from_zero():
    """SwiGLU of gates from -120 to 120, against 64 bits."""
    torch = _torch()
    K, I = 32, 64
    n = 241
    gate = torch.linspace(-120, 120, n, dtype=torch.float64)
    x = torch.zeros((n, K), device="cuda")
    x[:, 0], x[:, 1] = gate.float().cuda(), 3.0
    w = torch.full((1, 2 * I, K // 2), 0x88, dtype=torch.uint8, device="cuda")
    w[:, :I, 0] = 0x89  # gate rows: column 0 counts once
    w[:, I:, 0] = 0x98  # up rows: column 1
    y = binding.matmul_w4(x, w, torch.ones((1, 1, 2 * I), device="cuda"), swiglu=True, dtype=torch.float32)
    g64 = gate.float().double().cuda()
    want = (g64 * torch.sigmoid(g64) * 3.0)[:, None].expand(n, I)
    assert not bool(((y.double() - want).abs() > want.abs() * 18 * U + 2.0 ** -126).any())


def test_nothing_to_do():
    torch = _torch()
    w, scale, _ = weights(gen(1), 4, 64, 64, 32, False, "bf16", True)
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    y = binding.matmul_w4(torch.empty((0, 64), device="cuda"), w, scale, offsets=off)
    assert y.shape == (0, 64)
    y = torch.full((9, 64), 7.5, device="cuda")
    binding.matmul_w4(torch.zeros((9, 64), device="cuda"), w, scale, offsets=off, y=y)
    assert bool((y == 7.5).all())


@pytest.mark.parametrize("n", [40, 600])
def test_offsets_out_of_range(n):
    """Offsets before 0, past the rows and falling: rows that no expert can own stay as they were."""
    torch = _torch()
    w, scale, _ = weights(gen(2), 4, 64, 64, 32, False, "bf16", True)
    x = torch.ones((n, 64), device="cuda")
    y = torch.full((n + 8, 64), 7.5, device="cuda")
    off = torch.tensor([-5, 10, 20, n + 100, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    binding.matmul_w4(x, w, scale, offsets=off, y=y[:n])
    want, _, on = plain(x, w, scale, None, torch.tensor([0, 10, 20, n, n]))
    assert bool(on.all()) and torch.equal(y[:n], want.float())
    assert bool((y[n:] == 7.5).all())
    off = torch.tensor([10, 5, 30, 20, 35], dtype=torch.int32, device="cuda")
    y.fill_(7.5)
    binding.matmul_w4(x, w, scale, offsets=off, y=y[:n])
    assert bool((y[n:] == 7.5).all())


def test_codes_past_four_gib():
    """The last expert's codes lie more than 2^32 bytes behind the first's."""
    torch = _torch()
    E, M, K, G = 256, 2064, 16384, 128
    w = torch.zeros((E, M, K // 2), dtype=torch.uint8, device="cuda")
    g = gen(3)
    w[E - 1] = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.ones((E, K // G, M), dtype=torch.bfloat16, device="cuda")
    for n in (2, 80):
        x = torch.randint(-2, 3, (n, K), generator=g, device="cuda").to(torch.bfloat16)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[E] = n
        y = binding.matmul_w4(x, w, scale, offsets=off, dtype=torch.float32)
        want, _, _ = plain(x, w[E - 1:], scale[E - 1:], None, None)
        assert torch.equal(y, want.float())


@pytest.mark.parametrize("E,n,M,K", [(1, 3, 512, 1024), (64, 100, 256, 512), (16, 2000, 512, 512)])
def test_streams_and_repeats(E, n, M, K):
    """The same bits again, and on another stream."""
    torch = _torch()
    g = gen(n)
    w, scale, z = weights(g, E, M, K, 128, True, "bf16", False)
    x = torch.randn((n, K), generator=g, device="cuda").to(torch.bfloat16)
    off = None if E == 1 else split(n, E, 5)
    first = binding.matmul_w4(x, w, scale, zero=z, offsets=off, dtype=torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = [binding.matmul_w4(x, w, scale, zero=z, offsets=off, dtype=torch.float32, stream=side)
             for _ in range(3)]
    again = binding.matmul_w4(x, w, scale, zero=z, offsets=off, dtype=torch.float32)
    torch.cuda.synchronize()
    rows = slice(0, n) if off is None else slice(0, int(off[-1]))
    for y in other + [again]:
        assert torch.equal(y[rows], first[rows])


@pytest.mark.parametrize("E,n,M,K", [(1, 2, 1024, 2048), (32, 64, 256, 512), (8, 1500, 512, 512)])
def test_graph_replays(E, n, M, K):
    torch = _torch()
    g = gen(n)
    w, scale, _ = weights(g, E, M, K, 128, False, "bf16", False)
    x = torch.randn((n, K), generator=g, device="cuda").to(torch.bfloat16)
    off = None if E == 1 else split(n, E, 5)
    y = torch.zeros((n, M // 2), device="cuda")
    binding.matmul_w4(x, w, scale, offsets=off, swiglu=True, y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.matmul_w4(x, w, scale, offsets=off, swiglu=True, y=y)
    for i in range(5):
        x.copy_(torch.randn((n, K), generator=g, device="cuda"))
        y.zero_()
        graph.replay()
        got = y.clone()
        y.zero_()
        binding.matmul_w4(x, w, scale, offsets=off, swiglu=True, y=y)
        assert torch.equal(got, y), i


def test_gradients_are_refused():
    torch = _torch()
    w, scale, _ = weights(gen(4), 1, 64, 64, 32, False, "f32", False)
    x = torch.randn((4, 64), device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="no gradient"):
        binding.matmul_w4(x, w, scale)
    with pytest.raises(ValueError, match="no gradient"):
        binding.matmul_w4(x.detach(), w, scale.requires_grad_())
    with torch.no_grad():
        assert not binding.matmul_w4(x, w, scale).requires_grad
