"""GPU tests of the 4-bit products' block kernel, in every instance (w4_block_cases.py; a CPU test asks the choice
that each case runs there): what the tests of the few-row kernel hold for it too.

Whole numbers: rows, codes and zero points are whole and scales powers of two from 1/8 to 1, so that every sum is a whole
number of eighths below 2^24 of them (K |x| 255 8 < 2^24): fp32 holds every partial sum exactly in any order, fp32
results are equal to the 64-bit ones and bf16 results to their one rounding. SwiGLU: z is exact, silu is a few steps of
fp32 (taken as 16), the product one, and half a step of a bf16 result.
"""
import pytest

from sparse_moe_routing_amd import binding
from test_gpu_w4 import U, _torch, dt, gen, plain, swiglu_of, weights
from w4_block_cases import CASES, LARGE

pytestmark = pytest.mark.gpu

BEFORE, AFTER = 3, 5  # rows of no expert


class Case:
    def __init__(self, name, seed, whole=True, zeros=255):
        torch = _torch()
        counts, M, K, G, x, scale, zero, y, swiglu = CASES[name]
        g = gen(seed)
        self.dense, self.swiglu, self.K = len(counts) == 1, swiglu, K
        self.n = sum(counts) + (0 if self.dense else BEFORE + AFTER)
        self.w, self.scale, self.zero = weights(g, len(counts), M, K, G, zero, scale, whole)
        if zero and whole:
            self.zero = torch.randint(0, zeros + 1, self.zero.shape, generator=g, device="cuda").to(torch.uint8)
        xmax = max(1, min(9, (2 ** 21 - 1) // (K * 255)))
        if whole:
            self.x = torch.randint(-xmax, xmax + 1, (self.n, K), generator=g, device="cuda").to(dt(x))
        else:
            self.x = torch.randn((self.n, K), generator=g, device="cuda").to(dt(x))
        self.offsets = None
        if not self.dense:
            self.offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).int() + BEFORE
        self.ydt = dt(y)
        self.Mo = M // 2 if swiglu else M

    def run(self, x=None, y=None, **kw):
        if y is None and "dtype" not in kw:
            kw["dtype"] = self.ydt
        return binding.matmul_w4(self.x if x is None else x, self.w, self.scale, zero=self.zero, offsets=self.offsets,
                                 swiglu=self.swiglu, y=y, **kw)

    def rows(self):
        return slice(0, self.n) if self.dense else slice(BEFORE, self.n - AFTER)


def blank(c):
    torch = _torch()
    return torch.full((c.n, c.Mo), 7.5, dtype=c.ydt, device="cuda")


@pytest.mark.parametrize("name", CASES)
def test_whole_numbers(name):
    """Zero points up to 255; rows of no expert stay as they were."""
    torch = _torch()
    c = Case(name, 1)
    y = blank(c)
    assert c.run(y=y) is y
    want, _, on = plain(c.x, c.w, c.scale, c.zero, c.offsets)
    if c.swiglu:
        want = swiglu_of(want)
        half = 2.0 ** -8 * 1.01 if c.ydt is torch.bfloat16 else 0.0
        bad = (y.double() - want).abs() > want.abs() * (half + 18 * U) + 2.0 ** -126
        bad &= on[:, None]
    else:
        bad = (y != want.float().to(c.ydt)) & on[:, None]
    bad |= ~on[:, None] & (y != 7.5)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("name", CASES)
def test_infinities_stay_in_their_row(name):
    torch = _torch()
    c = Case(name, 2, zeros=15)
    clean = c.run(y=blank(c))
    first, last = c.rows().start, c.rows().stop - 1
    odd = [first, first + 20, (first + last) // 2, last - 1, last]
    x = c.x.clone()
    for i, n in enumerate(odd):
        x[n, (5 + 31 * i) % c.K] = float("nan") if i % 2 else float("inf")
    x[last, c.K - 1] = float("nan")
    y = c.run(x=x, y=blank(c))
    rest = torch.ones(c.n, dtype=torch.bool, device="cuda")
    rest[odd] = False
    assert torch.equal(y[rest], clean[rest])
    for i, n in enumerate(odd):
        if i % 2 or n == last:
            assert bool(y[n].isnan().all())
        elif not c.swiglu:  # inf times its weight: an infinity, or a NaN of weight 0
            assert not bool(y[n].isfinite().any())


@pytest.mark.parametrize("name", [n for n, c in CASES.items() if len(c[0]) > 1])
def test_rows_behind_the_last_are_not_read(name):
    """Rows of no expert that hold NaN, and a table that ends sooner: the other rows' bits stay."""
    torch = _torch()
    c = Case(name, 3)
    clean = c.run(y=blank(c))
    x = c.x.clone()
    x[:BEFORE] = x[-AFTER:] = float("nan")
    assert torch.equal(c.run(x=x, y=blank(c)), clean)
    end = int(c.offsets[-2])
    c.offsets[-1] = end + 1  # of the last expert's rows one is left
    y = c.run(x=x, y=blank(c))
    assert torch.equal(y[:end + 1], clean[:end + 1]) and bool((y[end + 1:] == 7.5).all())


@pytest.mark.parametrize("name", CASES)
def test_repeats_and_streams(name):
    """The same bits again, on another stream, and on two streams at once."""
    torch = _torch()
    c = Case(name, 4, whole=False)
    first = c.run(y=blank(c))
    side = [torch.cuda.Stream() for _ in range(2)]
    out = [blank(c) for _ in range(6)]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(3):
        for j, s in enumerate(side):
            c.run(y=out[2 * i + j], stream=s)
    again = c.run(y=blank(c))
    torch.cuda.synchronize()
    assert all(torch.equal(first, y) for y in out + [again])


@pytest.mark.parametrize("name", CASES)
def test_graph_replays(name):
    torch = _torch()
    c = Case(name, 5, whole=False)
    y = blank(c)
    c.run(y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(y=y)
    for i in range(3):
        c.x.copy_(torch.randn(c.x.shape, device="cuda"))
        if not c.dense:  # other rows per expert, read on the device
            c.offsets[1:-1] = torch.sort(torch.randint(BEFORE, c.n - AFTER + 1, c.offsets[1:-1].shape, device="cuda").int()).values
        y.fill_(7.5)
        graph.replay()
        got = y.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, c.run(y=blank(c))), i


def large(name):
    n, E, M, K, G, grouped, kw = LARGE[name]
    return n, E, M, K, G


def test_all_of_fp32_counts():
    """Rows whose elements use all 24 bits, against weights of 1: the gate's product is the row's element."""
    torch = _torch()
    n, _, M, K, G = large("all of fp32")
    g = gen(7)
    x = torch.zeros((n, K), device="cuda")
    at = torch.randint(0, K, (n,), generator=g, device="cuda")
    v = 1.0 + torch.randint(0, 2 ** 23, (n,), generator=g, device="cuda").double() / 2 ** 23
    x[torch.arange(n), at] = v.float()
    w = torch.full((1, M, K // 2), 0x99, dtype=torch.uint8, device="cuda")  # 9 - 8 = 1
    y = binding.matmul_w4(x, w, torch.ones((1, K // G, M), device="cuda"), dtype=torch.float32)
    assert torch.equal(y, v.float()[:, None].expand(n, M))


def test_every_code_and_zero():
    """One column at a time: code - zero of all 16 codes and of zeros from 0 to 255."""
    torch = _torch()
    n, _, M, K, G = large("every code and zero")
    x = torch.eye(K, device="cuda").to(torch.bfloat16).repeat(n // K, 1)
    zeros = (torch.arange(M, device="cuda") % 256).to(torch.uint8).reshape(1, 1, M).contiguous()
    w = torch.empty((1, M, K // 2), dtype=torch.uint8, device="cuda")
    w[:] = (torch.arange(16, device="cuda") | (torch.arange(16, device="cuda").flip(0) << 4)).to(torch.uint8)
    code = torch.stack([torch.arange(16), torch.arange(16).flip(0)], 1).reshape(-1).cuda().float().repeat(n // K)
    y = binding.matmul_w4(x, w, torch.ones((1, 1, M), device="cuda"), zero=zeros, dtype=torch.float32)
    assert torch.equal(y, code[:, None] - zeros.reshape(1, M).float())


def test_gates_far_from_zero():
    """SwiGLU of gates from -120 to 120, against 64 bits."""
    torch = _torch()
    n, _, M, K, G = large("gates")
    I = M // 2
    gate = torch.linspace(-120, 120, 241, dtype=torch.float64).repeat(n // 241)
    x = torch.zeros((n, K), device="cuda")
    x[:, 0], x[:, 1] = gate.float().cuda(), 3.0
    w = torch.full((1, M, K // 2), 0x88, dtype=torch.uint8, device="cuda")
    w[:, :I, 0] = 0x89  # gate rows: column 0 counts once
    w[:, I:, 0] = 0x98  # up rows: column 1
    y = binding.matmul_w4(x, w, torch.ones((1, 1, M), device="cuda"), swiglu=True, dtype=torch.float32)
    g64 = gate.float().double().cuda()
    want = (g64 * torch.sigmoid(g64) * 3.0)[:, None].expand(n, I)
    assert not bool(((y.double() - want).abs() > want.abs() * 18 * U + 2.0 ** -126).any())


def test_offsets_out_of_range():
    """Offsets before 0, past the rows and falling: rows that no expert can own stay as they were."""
    torch = _torch()
    n, E, M, K, G = large("offsets")
    w, scale, _ = weights(gen(2), E, M, K, G, False, "bf16", True)
    x = torch.ones((n, K), device="cuda")
    y = torch.full((n + 8, M), 7.5, device="cuda")
    off = torch.tensor([-5, 1000, 1020, n + 100, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    binding.matmul_w4(x, w, scale, offsets=off, y=y[:n])
    want, _, on = plain(x, w, scale, None, torch.tensor([0, 1000, 1020, n, n]))
    assert bool(on.all()) and torch.equal(y[:n], want.float())
    assert bool((y[n:] == 7.5).all())
    for falling in ([1000, 5, 2390, 20, 2395], [2400, 0, 2400, 0, 2400], [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0]):
        y.fill_(7.5)
        binding.matmul_w4(x, w, scale, offsets=torch.tensor(falling, dtype=torch.int32, device="cuda"), y=y[:n])
        assert bool((y[n:] == 7.5).all())


def test_codes_past_four_gib():
    """The last expert's codes lie more than 2^32 bytes behind the first's."""
    torch = _torch()
    n, E, M, K, G = large("codes past 4 GiB")
    w = torch.zeros((E, M, K // 2), dtype=torch.uint8, device="cuda")
    assert w.numel() // E * (E - 1) > 2 ** 32
    g = gen(3)
    w[E - 1] = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.ones((E, K // G, M), dtype=torch.bfloat16, device="cuda")
    x = torch.randint(-2, 3, (n, K), generator=g, device="cuda").to(torch.bfloat16)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = n
    y = binding.matmul_w4(x, w, scale, offsets=off)
    at = torch.randint(0, n, (300,), generator=g, device="cuda")
    want, _, _ = plain(x[at], w[E - 1:], scale[E - 1:], None, None)
    assert torch.equal(y[at], want.float().to(torch.bfloat16))


@pytest.mark.parametrize("name", ["rows past 4 GiB", "results past 4 GiB"])
def test_rows_past_four_gib(name):
    torch = _torch()
    n, _, M, K, G = large(name)
    assert n * max(M, K) * 2 > 2 ** 32
    g = gen(4)
    w, scale, _ = weights(g, 1, M, K, G, False, "bf16", True)
    x = torch.randint(-1, 2, (n, K), generator=g, device="cuda").to(torch.bfloat16)
    y = binding.matmul_w4(x, w, scale)
    for a in (0, n // 2, n - 200):
        want, _, _ = plain(x[a:a + 200], w, scale, None, None)
        assert torch.equal(y[a:a + 200], want.float().to(torch.bfloat16))
