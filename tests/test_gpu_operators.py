"""GPU parity of the separate operators (rows sorted by expert and back, their gradients, products
of 8-bit integers) against plain 64-bit forms computed here from the operators' definitions.

Tolerances count roundings. u = 2^-24 is half a step of fp32; a sum of n fp32 terms, each a rounded
product or a fused step, is off by at most n u sum|term| to first order (1.01 covers the rest);
the result is rounded once to its type, by at most eps / 2 of its value. Copies, codes, scales and
tables are compared exactly.
"""
import math

import pytest

from sparse_moe_routing_amd import binding

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -126


def _torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def half_step(dtype):
    return _torch().finfo(dtype).eps / 2


def check(got, want, bound, what):
    torch = _torch()
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float(err[bad].max()),
                                 bad.nonzero()[:3].tolist())


def routing(T, E, kept, seed, skew=False):
    """ids [T][8] of distinct experts; ids of experts outside [0, kept) belong to other shards."""
    torch = _torch()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = torch.randn((T, E), generator=g, device="cuda")
    if skew:
        z += 2.0 * torch.randn((E,), generator=g, device="cuda")
    top, ids = z.topk(8, dim=1)
    return ids.to(torch.int32), torch.softmax(top, 1), g


def tables(ids, kept):
    """(rows [T*8], offsets [kept + 1], kept pairs in sorted order) by a stable sort."""
    torch = _torch()
    flat = ids.reshape(-1).long()
    inside = (flat >= 0) & (flat < kept)
    order = torch.argsort(torch.where(inside, flat, torch.full_like(flat, kept)), stable=True)
    perm = order[:int(inside.sum())]
    rows = torch.full_like(flat, -1)
    rows[perm] = torch.arange(perm.numel(), device=flat.device)
    offsets = torch.zeros(kept + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = torch.bincount(flat[inside], minlength=kept).cumsum(0)
    return rows.to(torch.int32), offsets, perm


def types():
    torch = _torch()
    return {"f32": torch.float32, "bf16": torch.bfloat16}


# T, H, experts, experts of this shard, skewed: one token, odd counts, widths from one 16-byte
# piece to the largest and not a multiple of a wave's or a block's piece, shards that drop most
SHAPES = [(1, 8, 8, 8, False), (3, 24, 16, 16, False), (17, 200, 60, 15, True),
          (4, 2048, 256, 256, False), (257, 1000, 256, 32, True), (64, 4104, 255, 255, False),
          (33, 16384, 64, 8, False), (2050, 64, 256, 256, True), (700, 2048, 256, 256, False)]
DT = ["f32", "bf16"]


def dropped_table(rows, seed):
    """rows with more pairs dropped: every pair of token 0, and entries of all the kinds that
    mean it (-1, other negatives, the capacity, the largest int)."""
    torch = _torch()
    T8 = rows.numel()
    out = rows.clone()
    out[:8] = -1
    g = torch.Generator()
    g.manual_seed(seed)
    pick = torch.randperm(T8, generator=g)[:T8 // 5].cuda()
    kinds = torch.tensor([-1, -7, T8, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64, device="cuda")
    out[pick] = kinds[torch.arange(pick.numel(), device="cuda") % 5].to(torch.int32)
    return out


@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,H,E,kept,skew", SHAPES)
def test_permute(T, H, E, kept, skew, dt, dropped):
    torch = _torch()
    ids, _, g = routing(T, E, kept, 100 + T, skew)
    rows, _, _ = tables(ids, kept)
    if dropped:
        rows = dropped_table(rows, T)
    x = torch.randn((T, H), generator=g, device="cuda").to(types()[dt])
    x[0, 0] = float("nan")
    x[T - 1, H - 1] = float("-inf")
    xs = torch.full((T * 8, H), 7.5, dtype=x.dtype, device="cuda")
    want = xs.clone()
    r = rows.long()
    on = ((r >= 0) & (r < T * 8)).nonzero()[:, 0]
    want[r[on]] = x[on // 8]
    got = binding.permute(x, rows, xs=xs)
    assert got is xs
    as_bits = {"f32": torch.int32, "bf16": torch.int16}[dt]
    assert torch.equal(xs.view(as_bits), want.view(as_bits))  # rows of no pair as they were
    if not dropped:  # a smaller capacity drops the pairs past it and writes nothing there
        cap = max(1, int((rows >= 0).sum()) // 2)
        guard = torch.full((cap + 1, H), 7.5, dtype=x.dtype, device="cuda")
        binding.permute(x, rows, xs=guard[:cap])
        assert torch.equal(guard[:cap].view(as_bits), want[:cap].view(as_bits))
        assert bool((guard[cap] == 7.5).all())


@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,H,E,kept,skew", SHAPES)
def test_permute_backward(T, H, E, kept, skew, dt, dropped):
    torch = _torch()
    ids, _, g = routing(T, E, kept, 200 + T, skew)
    rows, _, _ = tables(ids, kept)
    if dropped:
        rows = dropped_table(rows, T)
    dxs = torch.randn((T * 8, H), generator=g, device="cuda").to(types()[dt])
    r = rows.long().reshape(T, 8)
    on = (r >= 0) & (r < T * 8)
    unused = torch.ones(T * 8, dtype=torch.bool, device="cuda")
    unused[r[on]] = False
    dxs[unused] = float("nan")  # rows of no pair are not read
    got = binding.permute_backward(dxs, rows)
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    for k in range(8):
        v = dxs.double()[r[:, k].clamp(0, T * 8 - 1)]
        v = torch.where(on[:, k, None], v, torch.zeros_like(v))
        want += v
        mag += v.abs()
    check(got, want, 1.01 * 8 * U * mag + half_step(got.dtype) * (want.abs() + 8 * U * mag), (T, H))
    gone = ~on.any(1)
    assert bool((got[gone] == 0).all())


def weighted(T, H, E, kept, skew, dt, out, shared, dropped, seed):
    torch = _torch()
    ids, w, g = routing(T, E, kept, seed + T, skew)
    rows, _, _ = tables(ids, kept)
    if dropped:
        rows = dropped_table(rows, T)
    r = rows.long().reshape(T, 8)
    on = (r >= 0) & (r < T * 8)
    w = torch.where(on, w, torch.full_like(w, float("nan")))  # a dropped pair's weight is not used
    ys = torch.randn((T * 8, H), generator=g, device="cuda").to(types()[dt])
    unused = torch.ones(T * 8, dtype=torch.bool, device="cuda")
    unused[r[on]] = False
    ys[unused] = float("nan")
    sh = gate = None
    if shared:
        sh = torch.randn((T, H), generator=g, device="cuda").to(types()[dt])
        gate = torch.sigmoid(torch.randn((T,), generator=g, device="cuda"))
    dy = torch.randn((T, H), generator=g, device="cuda").to(types()[out])
    return rows, r, on, w, ys, sh, gate, dy


@pytest.mark.parametrize("shared,dropped", [(False, False), (True, False), (False, True),
                                            (True, True)])
@pytest.mark.parametrize("dt,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"),
                                    ("bf16", "bf16")])
@pytest.mark.parametrize("T,H,E,kept,skew", SHAPES)
def test_unpermute(T, H, E, kept, skew, dt, out, shared, dropped):
    torch = _torch()
    rows, r, on, w, ys, sh, gate, _ = weighted(T, H, E, kept, skew, dt, out, shared, dropped, 300)
    y = torch.full((T + 1, H), 7.5, dtype=types()[out], device="cuda")
    binding.unpermute(ys, rows, w, shared=sh, gate=gate, y=y[:T])
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    for k in range(8):
        v = ys.double()[r[:, k].clamp(0, T * 8 - 1)] * w[:, k, None].double()
        v = torch.where(on[:, k, None], v, torch.zeros_like(v))
        want += v
        mag += v.abs()
    if shared:
        want += gate.double()[:, None] * sh.double()
        mag += (gate.double()[:, None] * sh.double()).abs()
    check(y[:T], want, 1.01 * 9 * U * mag + half_step(y.dtype) * (want.abs() + 9 * U * mag), (T, H))
    assert bool((y[T] == 7.5).all())


@pytest.mark.parametrize("shared,dropped", [(False, False), (True, False), (False, True),
                                            (True, True)])
@pytest.mark.parametrize("dt,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"),
                                    ("bf16", "bf16")])
@pytest.mark.parametrize("T,H,E,kept,skew", SHAPES)
def test_unpermute_backward(T, H, E, kept, skew, dt, out, shared, dropped):
    torch = _torch()
    rows, r, on, w, ys, sh, gate, dy = weighted(T, H, E, kept, skew, dt, out, shared, dropped, 400)
    dys0 = torch.full((T * 8, H), 7.5, dtype=ys.dtype, device="cuda")
    dys, dw, dsh, dg = binding.unpermute_backward(dy, ys, rows, w, shared=sh, gate=gate, dys=dys0)
    d = dy.double()
    named = torch.zeros(T * 8, dtype=torch.bool, device="cuda")
    named[r[on]] = True
    assert bool((dys[~named] == 7.5).all())
    hs = half_step(ys.dtype)
    # a dot product's longest chain: H terms at most, whatever the order
    n = H + 1
    for k in range(8):
        at = on[:, k].nonzero()[:, 0]
        want = w[at, k].double()[:, None] * d[at]
        check(dys[r[at, k]], want, (U + hs) * 1.01 * want.abs() + TINY, ("dys", T, H, k))
        prod = d[at] * ys[r[at, k]].double()
        check(dw[at, k], prod.sum(1), 1.01 * min(n, 2 ** 12) * U * prod.abs().sum(1), ("dw", T, H, k))
        assert bool((dw[~on[:, k], k] == 0).all())
    if shared:
        want = gate.double()[:, None] * d
        check(dsh, want, (U + hs) * 1.01 * want.abs() + TINY, ("dshared", T, H))
        prod = d * sh.double()
        check(dg, prod.sum(1), 1.01 * min(n, 2 ** 12) * U * prod.abs().sum(1), ("dgate", T, H))
    else:
        assert dsh is None and dg is None


def test_gradients_against_differences():
    """L = <c, y> is linear in each of ys, w, shared and gate, so a difference over a whole step
    is the directional derivative: it must equal the gradients' inner product with the step."""
    torch = _torch()
    T, H = 19, 136
    rows, r, on, w, ys, sh, gate, c = weighted(T, H, 32, 24, True, "f32", "f32", True, False, 900)
    w = torch.where(on, w, torch.zeros_like(w))
    ys = torch.where(torch.isnan(ys), torch.zeros_like(ys), ys)
    dys, dw, dsh, dg = binding.unpermute_backward(c, ys, rows, w, shared=sh, gate=gate,
                                                  dys=torch.zeros_like(ys))

    def loss(ys, w, sh, gate):
        return (c.double() * binding.unpermute(ys, rows, w, shared=sh, gate=gate).double()).sum()

    at = (ys, w, sh, gate)
    base = loss(*at)
    # each loss is a sum of 9 T H products, all of them below 64, with 10 roundings in each
    bound = 4 * 10 * U * 9 * T * H * 64 / math.sqrt(T * H)
    for i, grad in enumerate((dys, dw, dsh, dg)):
        step = torch.randn_like(at[i])
        step = torch.where(on, step, torch.zeros_like(step)) if i == 1 else step
        moved = list(at)
        moved[i] = at[i] + step
        got = loss(*moved) - base
        want = (grad.double() * (moved[i].double() - at[i].double())).sum()
        assert abs(float(got - want)) <= bound, (i, float(got), float(want))
    # and the sort with its gradient: <dxs, permute(x)> = <permute_backward(dxs), x>
    x = torch.randn((T, H), device="cuda")
    xs = binding.permute(x, rows, xs=torch.zeros((T * 8, H), device="cuda"))
    dxs = torch.randn((T * 8, H), device="cuda")
    lhs = (dxs.double() * xs.double()).sum()
    rhs = (binding.permute_backward(dxs, rows).double() * x.double()).sum()
    assert abs(float(lhs - rhs)) <= bound


# ----------------------------------------------------------------------------- 8-bit integers
def quantized(x):
    """(codes as float64, scales fp32) by the definition, in 64 bits."""
    torch = _torch()
    a = x.double().abs().amax(1)
    s = torch.where(a > 0, (a / 127.0).float(), torch.ones_like(a, dtype=torch.float32))
    s = s.clamp(min=TINY)
    return torch.round(x.double() / s.double()[:, None]), s


def rows_for_codes(n, K, dtype, seed):
    """Rows where rounding is decided by little: values on halves of the code grid and one step
    beside them, tiny and huge rows, a zero row."""
    torch = _torch()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((n, K), generator=g, device="cuda")
    if n > 1:  # multiples of half a code of a row whose maximum is 127, 254, ...: ties
        x[1] = torch.randint(-253, 254, (K,), generator=g, device="cuda") / 2.0
        x[1, 0] = 127.0
    if n > 2:
        x[2] = x[1] * 2.0 ** 100
    if n > 3:
        x[3] = 0.0
    if n > 4:
        x[4] *= 2.0 ** -130
    if n > 5:
        x[5] *= 2.0 ** -140
    if n > 6:
        x[6] = 1e38 * torch.sign(x[6])
    if n > 7:  # one step of the type off the halves
        x[7] = x[1] * (1.0 + 2.0 ** -8)
    if n > 8:  # half of the maximum: 63.5 codes
        x[8] = x[8, :1].abs() / 2 * torch.sign(x[8])
        x[8, 0] = 2 * x[8, 0]
    return x.to(dtype)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("n,K", [(1, 16), (9, 48), (12, 272), (40, 2048), (33, 4112), (10, 16384),
                                 (3000, 512)])
def test_quantize_i8(n, K, dt):
    torch = _torch()
    x = rows_for_codes(n, K, types()[dt], n + K)
    q, s = binding.quantize_i8(x)
    want_q, want_s = quantized(x)
    assert torch.equal(s, want_s)
    assert torch.equal(q.double(), want_q)
    assert int(q.min()) >= -127


def test_quantize_i8_not_finite():
    torch = _torch()
    for dt in types().values():
        x = torch.randn((5, 64), device="cuda").to(dt)
        x[1, 3] = float("nan")
        x[2, 63] = float("inf")
        x[3, 0] = float("-inf")
        q, s = binding.quantize_i8(x)
        assert bool(torch.isnan(s[1:4]).all()) and bool((q[1:4] == 0).all())
        w_q, w_s = quantized(x[[0, 4]])
        assert torch.equal(q[[0, 4]].double(), w_q) and torch.equal(s[[0, 4]], w_s)
        w = torch.ones((1, 8, 64), dtype=torch.int8, device="cuda")
        y = binding.matmul_i8(q, s, w, torch.ones((1, 8), device="cuda"), dtype=torch.float32)
        assert bool(torch.isnan(y[1:4]).all()) and bool(torch.isfinite(y[[0, 4]]).all())


@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,H,E,kept,skew", [(1, 16, 8, 8, False), (17, 208, 60, 15, True),
                                             (4, 2048, 256, 256, False), (257, 1008, 256, 32, True),
                                             (33, 16384, 64, 8, False), (2050, 64, 256, 256, True)])
def test_permute_i8(T, H, E, kept, skew, dt, dropped):
    torch = _torch()
    ids, _, _ = routing(T, E, kept, 500 + T, skew)
    rows, _, _ = tables(ids, kept)
    if dropped:
        rows = dropped_table(rows, T)
    x = rows_for_codes(T, H, types()[dt], T)
    q, s = binding.permute_i8(x, rows)
    want_q, want_s = quantized(x)
    r = rows.long()
    on = ((r >= 0) & (r < T * 8)).nonzero()[:, 0]
    assert torch.equal(q[r[on]].double(), want_q[on // 8])
    assert torch.equal(s[r[on]], want_s[on // 8])
    # rows of no pair are left alone: through the C entry into buffers with a mark
    mark_q = torch.full((T * 8, H), 99, dtype=torch.int8, device="cuda")
    mark_s = torch.full((T * 8,), 7.5, device="cuda")
    enum = binding.MOE_F32 if dt == "f32" else binding.MOE_BF16
    st = binding.load().moe_permute_i8(x.data_ptr(), rows.data_ptr(), T, H, T * 8, enum,
                                       mark_q.data_ptr(), mark_s.data_ptr(),
                                       torch.cuda.current_stream().cuda_stream)
    assert st == binding.MOE_OK
    named = torch.zeros(T * 8, dtype=torch.bool, device="cuda")
    named[r[on]] = True
    assert bool((mark_q[~named] == 99).all()) and bool((mark_s[~named] == 7.5).all())
    assert torch.equal(mark_q[named], q[named]) and torch.equal(mark_s[named], s[named])


def i8_case(n, K, M, E, seed):
    torch = _torch()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randint(-127, 128, (n, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (E, M, K), generator=g, device="cuda", dtype=torch.int8)
    # scales that give products of about 1, some rows and channels far from it
    xs = torch.rand((n,), generator=g, device="cuda") * 2e-2 + 1e-3
    ws = (torch.rand((E, M), generator=g, device="cuda") * 2e-2 + 1e-3) / math.sqrt(K)
    return x, xs, w, ws


def i8_check(y, x, xs, w, ws, lo, hi, e, swiglu, what):
    """Rows lo..hi of y, expert e's. z: the fp32 value of the integer sum and two products, three
    roundings; SwiGLU: an error of 3 u in the gate moves silu by at most 3 (1 + |gate|) u, its
    exponential (2 steps), sum, quotient and the product with up (3 u, one more) add 10 u."""
    torch = _torch()
    z = (x[lo:hi].double() @ w[e].double().t().contiguous()) * xs[lo:hi].double()[:, None] * \
        ws[e].double()[None, :]
    hs = half_step(y.dtype)
    if swiglu:
        g, u = z[:, :z.shape[1] // 2], z[:, z.shape[1] // 2:]
        z = g * torch.sigmoid(g) * u
        rel = (3 * (1 + g.abs()) + 10) * U
    else:
        rel = 3 * U
    check(y[lo:hi], z, 1.01 * (rel + hs) * z.abs() + 1e-36, what)


# counts of each expert's rows: empty experts at both ends and between, one row, one past and
# one short of row tiles, more than a tile
COUNTS = [[1], [0, 1, 0], [4, 0, 15, 16, 17, 0, 0, 31, 33], [63, 64, 65, 0, 1], [0, 0, 200, 0],
          [129, 255, 257, 1, 0, 320, 321, 511]]


@pytest.mark.parametrize("out", DT)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K,M", [(16, 16), (64, 48), (208, 272), (2048, 144), (512, 2048),
                                 (1040, 1024), (16384, 32)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "_".join(map(str, c)))
def test_matmul_i8_grouped(counts, K, M, swiglu, out):
    torch = _torch()
    E, first, tail = len(counts), 3, 5  # rows before the first expert's and behind the last's
    n = first + sum(counts) + tail
    x, xs, w, ws = i8_case(n, K, M, E, 7 + K + M)
    offsets = torch.tensor([first] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    Mo = M // 2 if swiglu else M
    y = torch.full((n, Mo), 7.5, dtype=types()[out], device="cuda")
    binding.matmul_i8(x, xs, w, ws, offsets=offsets, swiglu=swiglu, y=y)
    lo = first
    for e, c in enumerate(counts):
        if c:
            i8_check(y, x, xs, w, ws, lo, lo + c, e, swiglu, (counts, K, M, e))
        lo += c
    assert bool((y[:first] == 7.5).all()) and bool((y[lo:] == 7.5).all())


@pytest.mark.parametrize("out", DT)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("n,K,M", [(1, 2048, 1024), (2, 16, 16), (4, 512, 2048), (5, 48, 80),
                                   (16, 4096, 96), (17, 2064, 528), (100, 1008, 1040),
                                   (513, 320, 560), (1025, 2048, 1024), (2049, 1024, 4096)])
def test_matmul_i8_dense(n, K, M, swiglu, out):
    x, xs, w, ws = i8_case(n, K, M, 1, n)
    y = binding.matmul_i8(x, xs, w, ws, swiglu=swiglu, dtype=types()[out])
    i8_check(y, x, xs, w, ws, 0, n, 0, swiglu, (n, K, M))


# enough rows that blocks of 128 or 320 rows multiply them: K of 1 to 8 slabs of 128, whole and not,
# M in whole and partial channel blocks, tiles of 1 row to the full block
MANY = {"long": [20011, 0, 9000, 999, 1], "medium": [(37 * i) % 181 for i in range(96)]}


@pytest.mark.parametrize("out", DT)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K,M", [(16, 1040), (144, 1552), (256, 528), (272, 2048), (400, 1296),
                                 (512, 272), (656, 1040), (784, 1024), (1008, 784)])
@pytest.mark.parametrize("counts", list(MANY))
def test_matmul_i8_many_rows(counts, K, M, swiglu, out):
    torch = _torch()
    counts = MANY[counts]
    E, n = len(counts), sum(counts) + 2
    x, xs, w, ws = i8_case(n, K, M, E, K + M)
    offsets = torch.tensor([1] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    y = torch.full((n, M // 2 if swiglu else M), 7.5, dtype=types()[out], device="cuda")
    binding.matmul_i8(x, xs, w, ws, offsets=offsets, swiglu=swiglu, y=y)
    lo = 1
    for e, c in enumerate(counts):
        if c:
            i8_check(y, x, xs, w, ws, lo, lo + c, e, swiglu, (K, M, e))
        lo += c
    assert bool((y[0] == 7.5).all()) and bool((y[lo:] == 7.5).all())


@pytest.mark.parametrize("out", DT)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("n,K,M", [(1000, 144, 4112), (700, 272, 4096), (513, 400, 8208),
                                   (2100, 656, 4112), (30001, 144, 1040), (20480, 272, 2064),
                                   (16001, 1008, 1040), (9999, 128, 4096)])
def test_matmul_i8_dense_many_rows(n, K, M, swiglu, out):
    x, xs, w, ws = i8_case(n, K, M, 1, n)
    y = binding.matmul_i8(x, xs, w, ws, swiglu=swiglu, dtype=types()[out])
    i8_check(y, x, xs, w, ws, 0, n, 0, swiglu, (n, K, M))


@pytest.mark.parametrize("T,E,K,M,swiglu", [(1, 256, 512, 256, True), (4, 256, 2048, 1024, True),
                                            (32, 256, 512, 2048, False), (192, 255, 256, 512, True),
                                            (300, 60, 1024, 272, False), (1030, 16, 512, 1024, True),
                                            (4097, 64, 512, 512, False)])
def test_matmul_i8_routed(T, E, K, M, swiglu):
    """Every expert of a routed round, and the same bits when an expert's rows come alone."""
    torch = _torch()
    ids, _, _ = routing(T, E, E, 600 + T, True)
    rows, offsets, perm = tables(ids, E)
    n = T * 8
    x, xs, w, ws = i8_case(n, K, M, E, T)
    y = binding.matmul_i8(x, xs, w, ws, offsets=offsets, swiglu=swiglu, dtype=torch.float32)
    o = offsets.tolist()
    alone = 0
    for e in range(E):
        if o[e] == o[e + 1]:
            continue
        i8_check(y, x, xs, w, ws, o[e], o[e + 1], e, swiglu, (T, e))
        if alone < 3:
            alone += 1
            one = binding.matmul_i8(x[o[e]:o[e + 1]].contiguous(), xs[o[e]:o[e + 1]].contiguous(),
                                    w[e:e + 1], ws[e:e + 1].contiguous(), swiglu=swiglu,
                                    dtype=torch.float32)
            assert torch.equal(one, y[o[e]:o[e + 1]])


def test_matmul_i8_extreme_codes():
    """All codes at their largest magnitude at the largest K: 2^28 in the 32-bit sum."""
    torch = _torch()
    K = 16384
    for a, b in ((127, 127), (-128, -128), (127, -128)):
        x = torch.full((20, K), a, dtype=torch.int8, device="cuda")
        w = torch.full((1, 32, K), b, dtype=torch.int8, device="cuda")
        y = binding.matmul_i8(x, torch.ones(20, device="cuda"), w, torch.ones((1, 32), device="cuda"),
                              dtype=torch.float32)
        assert bool((y == float(a * b * K)).all())


def test_offsets_out_of_order_stay_inside():
    """Offsets past the rows are clamped, and where they fall nothing outside y is touched. Here expert 0 has rows 0..9 (from -5), experts 1 and
    2 none (10..10, 10..8), expert 3 rows 8..39: rows 8 and 9 are in two ranges, and either
    expert's."""
    torch = _torch()
    n, K, M = 40, 64, 32
    x, xs, w, ws = i8_case(n, K, M, 4, 5)
    buf = torch.full((n + 64, M), 7.5, device="cuda")
    offsets = torch.tensor([-5, 10, 10, 8, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    binding.matmul_i8(x, xs, w, ws, offsets=offsets, y=buf[:n])
    i8_check(buf, x, xs, w, ws, 0, 8, 0, False, "first")
    i8_check(buf, x, xs, w, ws, 10, n, 3, False, "last")
    assert bool((buf[n:] == 7.5).all())


# ----------------------------------------------------------------------------- sizes past 32 bits
def test_rows_past_32_bits():
    """Sorted buffers of more than 2^32 bytes and 2^31 elements: rows at their far end."""
    torch = _torch()
    H, T = 16384, 2
    n = 2 ** 31 // H + 4096
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    r = torch.tensor([n - 1 - 7 * i for i in range(16)], dtype=torch.int32, device="cuda")
    r[3] = -1
    keep = [i for i in range(16) if i != 3]
    xs = torch.empty((n, H), dtype=torch.bfloat16, device="cuda")
    binding.permute(x, r, xs=xs)
    for i in keep:
        assert torch.equal(xs[int(r[i])], x[i // 8])
    w = torch.softmax(torch.randn((T, 8), device="cuda"), 1)
    y = binding.unpermute(xs, r, w, dtype=torch.float32)
    ww = w.double()
    ww[0, 3] = 0
    want = ww.sum(1)[:, None] * x.double()
    check(y, want, 1.01 * 9 * U * want.abs() + U * want.abs(), "far rows")
    dx = binding.permute_backward(xs, r)
    cnt = torch.tensor([7.0, 8.0], device="cuda", dtype=torch.float64)[:, None]
    check(dx, cnt * x.double(), (8 * U + half_step(dx.dtype)) * 1.01 * cnt * x.double().abs(), "dx")
    dy = torch.randn((T, H), device="cuda")
    dys, dw, _, _ = binding.unpermute_backward(dy, xs, r, w, dys=torch.empty_like(xs))
    for i in keep:
        want = w[i // 8, i % 8].double() * dy[i // 8].double()
        check(dys[int(r[i])], want, (U + 2.0 ** -8) * 1.01 * want.abs(), "far dys")
    assert float(dw[0, 3]) == 0.0
    del xs, dys
    q, s = binding.permute_i8(x, r, n_rows=n)
    want_q, want_s = quantized(x)
    for i in keep:
        assert torch.equal(q[int(r[i])].double(), want_q[i // 8]) and s[int(r[i])] == want_s[i // 8]


def test_matmul_i8_past_32_bits():
    """Weights past 2^31 bytes, rows and results past 2^31 elements: the last expert's last rows."""
    torch = _torch()
    E, M, K = 130, 1024, 16384
    w = torch.empty((E, M, K), dtype=torch.int8, device="cuda")
    w[E - 1] = torch.randint(-127, 128, (M, K), device="cuda", dtype=torch.int8)
    ws = torch.full((E, M), 1e-3, device="cuda")
    n = 2 ** 31 // M + 1000
    x = torch.empty((n, K), dtype=torch.int8, device="cuda")
    x[n - 70:] = torch.randint(-127, 128, (70, K), device="cuda", dtype=torch.int8)
    xs = torch.full((n,), 1e-3, device="cuda")
    offsets = torch.full((E + 1,), n - 70, dtype=torch.int32, device="cuda")
    offsets[E] = n
    y = torch.empty((n, M), dtype=torch.float32, device="cuda")
    binding.matmul_i8(x, xs, w, ws, offsets=offsets, y=y)
    i8_check(y, x, xs, w, ws, n - 70, n, E - 1, False, "far rows")


def test_largest_counts():
    """The most tokens, rows and channels the entry points take, at the narrowest widths."""
    torch = _torch()
    T, H = 1048576, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    rows = torch.randperm(T * 8, generator=g, device="cuda").to(torch.int32)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    src = torch.empty(T * 8, dtype=torch.long, device="cuda")
    src[rows.long()] = torch.arange(T * 8, device="cuda") // 8
    xs = binding.permute(x, rows)
    assert torch.equal(xs, x[src])
    dx = binding.permute_backward(xs, rows)
    assert torch.equal(dx, (x.double() * 8).to(torch.bfloat16))  # eight equal terms: exact
    w = torch.full((T, 8), 0.125, device="cuda")
    y = binding.unpermute(xs, rows, w, dtype=torch.float32)
    assert torch.equal(y, x.float())  # eighths: exact
    dys, dw, _, _ = binding.unpermute_backward(y, xs, rows, w)
    assert torch.equal(dys, (xs.float() * 0.125).to(torch.bfloat16))
    want = (x.double() ** 2).sum(1, keepdim=True).expand(T, 8)
    check(dw, want, 1.01 * H * U * want, "dw")
    q, s = binding.permute_i8(x, rows)
    want_q, want_s = quantized(x)
    assert torch.equal(q.double(), want_q[src]) and torch.equal(s, want_s[src])
    q2, s2 = binding.quantize_i8(xs)
    assert torch.equal(q2, q) and torch.equal(s2, s)
    wq = torch.randint(-127, 128, (2, 8, H), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.full((2, 8), 0.01, device="cuda")
    n = T * 8
    offsets = torch.tensor([0, n - 5, n], dtype=torch.int32, device="cuda")
    y = binding.matmul_i8(q, s, wq, ws, offsets=offsets, dtype=torch.float32)
    i8_check(y, q, s, wq, ws, 0, n - 5, 0, False, "all but five")
    i8_check(y, q, s, wq, ws, n - 5, n, 1, False, "five")
    for rows_n in (3, 700):
        x8, xs8, w8, ws8 = i8_case(rows_n, 32, 65536, 1, 3)
        i8_check(binding.matmul_i8(x8, xs8, w8, ws8, swiglu=True), x8, xs8, w8, ws8, 0, rows_n, 0, True, "wide")


# ----------------------------------------------------------------------------- tables
@pytest.mark.parametrize("T", [1, 7, 8, 9, 33, 64, 65, 200, 256, 257, 1000, 4097])
def test_bucket_rows(T):
    """The tables of moe_bucket bit for bit, and rows the inverse of perm; dropped pairs -1."""
    torch = _torch()
    from sparse_moe_routing_amd import inputs
    layer = inputs.make_layer(inputs.BY_NAME["tiny_fp32_t4"])
    m, _ = binding.layer_from_numpy(layer, 8192)
    E = m.num_experts
    ids, _, g = routing(T, E, E, 800 + T)
    some = torch.rand(ids.shape, generator=g, device="cuda") < 0.1
    ids = torch.where(some, ids - 2 * E, ids)
    if T > 2:
        ids[2] = E  # a token without a kept pair
    ws = m.workspace(T)
    counts, offsets, perm, rows = m.bucket_rows(ids, ws=ws)
    c0, o0, p0 = m.bucket(ids, ws=ws)
    n = int(offsets[E])
    assert torch.equal(counts, c0) and torch.equal(offsets, o0) and torch.equal(perm[:n], p0[:n])
    want_rows, want_offsets, want_perm = tables(ids, E)
    assert torch.equal(rows, want_rows) and torch.equal(offsets, want_offsets)
    assert torch.equal(perm[:n].long(), want_perm)
    assert bool((ws[:m.state_bytes()] == 0).all())
    m.close()


# ----------------------------------------------------------------------------- used together
def bf16_weights(w, scale):
    return (w.double() * scale.double()[..., None]).to(_torch().bfloat16)


@pytest.mark.parametrize("T", [1, 4, 33, 192, 1000])
def test_int8_layer(T):
    """The layer with 8-bit integer experts as a serving loop runs it: route, bucket, sort with
    quantisation, gate/up with SwiGLU, quantise, down, return with weights and the gated shared
    expert. Each step against its 64-bit form on the step's own inputs, and y against the layer's
    bf16 experts of the decoded weights within what 8 bits of activations leave."""
    torch = _torch()
    H, E, I, Is = 512, 32, 256, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(40 + T)

    def codes(*shape):
        v = torch.randn(shape, generator=g, device="cuda") / math.sqrt(shape[-1])
        s = v.abs().amax(-1) / 127
        return torch.round(v / s[..., None]).to(torch.int8), s

    gu, gus = codes(E, 2 * I, H)
    dn, dns = codes(E, H, I)
    sgu, sgus = codes(1, 2 * Is, H)
    sdn, sdns = codes(1, H, Is)
    weights = {"router_w": (torch.randn((E + 1, H), generator=g, device="cuda") / math.sqrt(H)).to(
        torch.bfloat16), "gate_up": bf16_weights(gu, gus), "down": bf16_weights(dn, dns),
        "shared_gate_up": bf16_weights(sgu, sgus)[0].contiguous(),
        "shared_down": bf16_weights(sdn, sdns)[0].contiguous()}
    m = binding.MoeLayer(H, E, I, Is, 1024, "bf16", weights)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ws = m.workspace(T)
    _, ids, w, gate = m.route(x=x, ws=ws, want_logits=False)
    counts, offsets, perm, rows = m.bucket_rows(ids, ws=ws)
    q, qs = binding.permute_i8(x, rows)
    h = binding.matmul_i8(q, qs, gu, gus, offsets=offsets, swiglu=True)
    hq, hqs = binding.quantize_i8(h)
    ys = binding.matmul_i8(hq, hqs, dn, dns, offsets=offsets)
    sq, sqs = binding.quantize_i8(x)
    sh = binding.matmul_i8(sq, sqs, sgu, sgus, swiglu=True)
    shq, shqs = binding.quantize_i8(sh)
    shared = binding.matmul_i8(shq, shqs, sdn, sdns)
    y = binding.unpermute(ys, rows, w, shared=shared, gate=gate, dtype=torch.float32)
    # step by step
    want_rows, want_offsets, want_perm = tables(ids, E)
    assert torch.equal(rows, want_rows) and torch.equal(offsets, want_offsets)
    xq, xs = quantized(x)
    assert torch.equal(q.double(), xq[want_perm // 8]) and torch.equal(qs, xs[want_perm // 8])
    o = offsets.tolist()
    for e in range(E):
        if o[e + 1] > o[e]:
            i8_check(h, q, qs, gu, gus, o[e], o[e + 1], e, True, ("h", e))
            i8_check(ys, hq, hqs, dn, dns, o[e], o[e + 1], e, False, ("ys", e))
    for got_q, got_s, src in ((hq, hqs, h), (sq, sqs, x), (shq, shqs, sh)):
        want_q, want_s = quantized(src)
        assert torch.equal(got_q.double(), want_q) and torch.equal(got_s, want_s)
    i8_check(sh, sq, sqs, sgu, sgus, 0, T, 0, True, "shared h")
    i8_check(shared, shq, shqs, sdn, sdns, 0, T, 0, False, "shared")
    r = rows.long().reshape(T, 8)
    terms = torch.cat([w.double()[:, :, None] * ys.double()[r],
                       (gate.double()[:, None] * shared.double())[:, None]], 1)
    check(y, terms.sum(1), 1.01 * 10 * U * terms.abs().sum(1), "y")
    # against the layer's own bf16 path on the decoded weights (each rounded to bf16: 2^-9 of its
    # value in the mean): the activations' codes are off by up to half a code of ~40 codes' rms,
    # 0.29 / 40 in the mean, twice (x and h), so 1 % of |y|_2 each; 4 % is twice their sum
    y_ref = m.forward(x, routing=(ids, w, gate), ws=ws)
    rel = float((y.double() - y_ref.double()).norm() / y_ref.double().norm())
    assert rel <= 0.04, rel
    m.close()


def test_training_step():
    """Sort, a caller's own expert product (fp32, torch), return: outputs and every gradient of
    the two operators against autograd in 64 bits."""
    torch = _torch()
    T, H, E, kept = 37, 72, 16, 12
    ids, w, g = routing(T, E, kept, 71)
    rows, offsets, perm = tables(ids, kept)
    N = perm.numel()
    x = torch.randn((T, H), generator=g, device="cuda")
    we = torch.randn((kept, H, H), generator=g, device="cuda") / math.sqrt(H)
    sh = torch.randn((T, H), generator=g, device="cuda")
    gate = torch.sigmoid(torch.randn((T,), generator=g, device="cuda"))
    dy = torch.randn((T, H), generator=g, device="cuda")
    o = offsets.tolist()

    def experts(xs, weights):
        return torch.cat([xs[o[e]:o[e + 1]] @ weights[e] for e in range(kept)])

    xs = binding.permute(x, rows, n_rows=N)
    ys = experts(xs.double(), we.double()).float()
    y = binding.unpermute(ys, rows, w, shared=sh, gate=gate)
    dys, dw, dsh, dg = binding.unpermute_backward(dy, ys, rows, w, shared=sh, gate=gate)
    dxs = torch.cat([dys[o[e]:o[e + 1]].double() @ we[e].double().t().contiguous()
                     for e in range(kept)]).float()
    dx = binding.permute_backward(dxs, rows)
    X, W, S, G = (t.double().cpu().requires_grad_() for t in (x, w, sh, gate))
    pc = perm.cpu()
    Ys = experts(X[pc // 8], we.double().cpu())
    Y = torch.zeros((T, H), dtype=torch.float64).index_add(0, pc // 8, Ys * W.reshape(-1)[pc][:, None])
    Y = Y + G[:, None] * S
    Y.backward(dy.double().cpu())
    # each value is a sum of at most 9 H products of fp32-rounded numbers
    for got, want in ((y, Y.detach()), (dx, X.grad), (dw, W.grad), (dsh, S.grad), (dg, G.grad)):
        want = want.cuda()
        scale = float(want.abs().max())
        check(got, want, torch.full_like(want, 9 * math.sqrt(H) * 4 * U * scale), "training")


# ----------------------------------------------------------------------------- streams and graphs
def one_of_each(seed, T=70, H=512, E=32, I=128):
    torch = _torch()
    ids, w, g = routing(T, E, E, seed)
    rows, offsets, perm = tables(ids, E)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    gu = torch.randint(-127, 128, (E, 2 * I, H), generator=g, device="cuda", dtype=torch.int8)
    gus = torch.full((E, 2 * I), 4e-4, device="cuda")
    dn = torch.randint(-127, 128, (E, H, I), generator=g, device="cuda", dtype=torch.int8)
    dns = torch.full((E, H), 8e-4, device="cuda")
    dy = torch.randn((T, H), generator=g, device="cuda")

    def step(stream=None):
        k = {} if stream is None else {"stream": stream}
        xs = binding.permute(x, rows, **k)
        q, qs = binding.permute_i8(x, rows, **k)
        h = binding.matmul_i8(q, qs, gu, gus, offsets=offsets, swiglu=True, **k)
        hq, hqs = binding.quantize_i8(h, **k)
        ys = binding.matmul_i8(hq, hqs, dn, dns, offsets=offsets, **k)
        y = binding.unpermute(ys, rows, w, dtype=torch.float32, **k)
        dys, dw, _, _ = binding.unpermute_backward(dy, ys, rows, w, **k)
        dx = binding.permute_backward(dys, rows, **k)
        return [xs, q, qs, h, ys, y, dys, dw, dx]

    return x, step


def test_side_stream():
    torch = _torch()
    x, step = one_of_each(81)
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once():
    torch = _torch()
    (_, a), (_, b) = one_of_each(82), one_of_each(83, T=300)
    want = a(), b()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(3):
        for i, f in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(f())
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(run, want[i]))


@pytest.mark.parametrize("T", [4, 700])
def test_graph_capture_replays(T):
    """Two captured graphs of all operators, replayed in turn with new inputs and eager calls
    between, give the eager results bit for bit."""
    torch = _torch()
    made = [one_of_each(84 + i, T=T) for i in range(2)]
    graphs = []
    for x, step in made:
        step()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step()
        graphs.append((gr, out))
    for r in range(3):
        for (x, step), (gr, out) in zip(made, graphs):
            x.copy_(torch.randn_like(x, dtype=torch.float32).to(x.dtype))
            for t in out:
                t.zero_()
            gr.replay()
            torch.cuda.synchronize()
            want = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), r


def test_operands_side_by_side():
    """Operands that touch in one allocation are no overlap; one byte more in common is refused."""
    torch = _torch()
    T, H = 5, 64
    rows = tables(routing(T, 16, 16, 90)[0], 16)[0]
    room = torch.zeros((T + 8 * T + T, H), device="cuda")
    x, xs, dx = room[:T], room[T:9 * T], room[9 * T:]
    x.copy_(torch.randn(T, H, device="cuda"))
    want = binding.permute(x, rows)
    assert torch.equal(binding.permute(x, rows, xs=xs), want)
    assert torch.equal(binding.permute_backward(xs, rows, dx=dx), binding.permute_backward(want, rows))
    w = torch.full((T, 8), 0.125, device="cuda")
    assert torch.equal(binding.unpermute(xs, rows, w, y=dx), binding.unpermute(want, rows, w))
    before = room.clone()
    for bad in (lambda: binding.permute(x, rows, xs=room[T - 1:9 * T - 1]),
                lambda: binding.permute_backward(xs, rows, dx=room[9 * T - 1:10 * T - 1]),
                lambda: binding.unpermute(xs, rows, w, y=room[9 * T - 1:10 * T - 1]),
                lambda: binding.unpermute_backward(x, xs, rows, w, dys=xs)):
        with pytest.raises(binding.MoeError):
            bad()
    torch.cuda.synchronize()
    assert torch.equal(room, before)


def test_bucket_rows_without_tokens():
    torch = _torch()
    from sparse_moe_routing_amd import inputs
    m, _ = binding.layer_from_numpy(inputs.make_layer(inputs.BY_NAME["tiny_fp32_t4"]), 64)
    ids = torch.empty((0, 8), dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    for s in (None, side):
        counts, offsets, perm, rows = m.bucket_rows(ids, stream=s)
        torch.cuda.synchronize()
        assert not counts.any() and not offsets.any() and perm.numel() == rows.numel() == 0
    m.close()
