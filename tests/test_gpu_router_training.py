"""GPU tests of what trains the router: the balance loss with its counts and gradient, and the
gradient of the selection's weights, against 64-bit forms computed here.

u = 2^-24. A probability: the logit's difference a to the row's largest is rounded (u |a|), times
log2(e) (rounded: u |a|; the constant's own error: less than u |a| / 2), 2^x and the reciprocal are
within 2u, the sum of E <= 256 terms runs in at most 16 + 4 additions, the product adds u: relative error
at most REL = (2.5 A + 30) u, with A the largest difference. Probabilities below 2^-126 may be 0.
"""
import pytest

from sparse_moe_routing_amd import binding, inputs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def gen(seed):
    torch = _torch()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def dt(name):
    torch = _torch()
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def case(T, E, R, dtype, masked, seed, odd_ids=False):
    torch = _torch()
    g = gen(seed)
    z = torch.randn((T, R), generator=g, device="cuda") * 2
    ids = z[:, :E].topk(8, dim=1).indices.to(torch.int32)
    if odd_ids and T:
        pick = torch.randint(0, T * 8, (T,), generator=g, device="cuda")
        kinds = torch.tensor([-1, E, E + 3, -2 ** 31, 2 ** 31 - 1, 0, 0], dtype=torch.int64, device="cuda")
        ids.view(-1)[pick] = kinds[torch.arange(T, device="cuda") % 7].to(torch.int32)
    mask = None
    if masked == "some":
        mask = torch.rand((T,), generator=g, device="cuda") < 0.6
    elif masked == "none left":
        mask = torch.zeros((T,), dtype=torch.bool, device="cuda")
    return z.to(dt(dtype)), ids, mask


def plain(z, ids, E, mask):
    """(P, counts, N, f) in 64 bits; rows that do not count are left out of P (0)."""
    torch = _torch()
    T = z.shape[0]
    on = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    s = z[:, :E].double()
    m = s.amax(1, keepdim=True) if T else s
    none = m == float("-inf")
    e = torch.exp(s - torch.where(none, torch.zeros_like(m), m))
    p = torch.where(none, torch.zeros_like(e), e / e.sum(1, keepdim=True))
    p = torch.where(on[:, None], p, torch.zeros_like(p))
    flat = ids[on].reshape(-1).long()
    counts = torch.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
    n = int(on.sum())
    f = counts.double() / (8 * max(n, 1))
    return p, counts, n, f


def check(z, ids, E, mask, spread=20.0):
    torch = _torch()
    rel = (2.5 * spread + 30) * U
    p, counts, n, f = plain(z, ids, E, mask)
    loss, c, tokens = binding.balance_loss(z, ids, E, mask=mask)
    assert loss.shape == () and tokens.shape == () and tokens.dtype == c.dtype == torch.int32
    assert torch.equal(c.long(), counts) and int(tokens) == n
    want = E * float((f * p.sum(0)).sum()) / max(n, 1)
    # the tokens' sums: at most 64 in a lane, 2 across lanes, one rounding a block and of the result
    assert abs(float(loss) - want) <= want * (rel + 70 * U), (float(loss), want)
    dloss = torch.tensor(0.37, device="cuda")
    dz = binding.balance_loss_backward(dloss, z, c, tokens, mask=mask)
    assert dz.dtype == z.dtype and dz.shape == z.shape
    if z.shape[0] == 0:
        return
    k = float(dloss.double()) * E / max(n, 1)
    d = f - (1.0 / E if n else 0.0)
    centre = (p * d).sum(1, keepdim=True)
    size = p * (d.abs()[None, :] + (p * d.abs()).sum(1, keepdim=True))
    want = torch.zeros(z.shape, dtype=torch.float64, device="cuda")
    # for a row of probabilities that sum to 1; the rows without any have gradient 0 in both forms
    want[:, :E] = k * p * (d - centre)
    half = torch.finfo(z.dtype).eps / 2
    bound = torch.zeros_like(want)
    bound[:, :E] = k * size * (2 * rel + 30 * U) * 1.01
    bound += half * want.abs() + 2.0 ** -126
    bad = (dz.double() - want).abs() > bound
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:3].tolist())
    if mask is not None:
        assert bool((dz[~mask.bool()] == 0).all())
    assert bool((dz[:, E:] == 0).all())


SHAPES = [(0, 16, 17), (1, 8, 8), (1, 256, 257), (3, 9, 16), (4, 64, 65), (5, 65, 65), (63, 128, 128),
          (64, 129, 130), (65, 255, 256), (192, 256, 257), (511, 60, 61), (513, 16, 17), (2050, 256, 256),
          (8192, 256, 257), (33000, 64, 64)]


@pytest.mark.parametrize("masked", ["no", "some", "none left"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,R", SHAPES)
def test_balance(T, E, R, dtype, masked):
    z, ids, mask = case(T, E, R, dtype, masked, 10 + T)
    check(z, ids, E, mask)


@pytest.mark.parametrize("masked", ["no", "some"])
@pytest.mark.parametrize("T", [1, 70, 3000])
def test_balance_ids_outside_and_repeated(T, masked):
    z, ids, mask = case(T, 60, 61, "f32", masked, T, odd_ids=True)
    check(z, ids, 60, mask)


def test_balance_of_an_even_routing_is_one():
    torch = _torch()
    E = 32
    z = torch.zeros((64, E), device="cuda")
    ids = (torch.arange(64 * 8, device="cuda") % E).reshape(64, 8).to(torch.int32)
    loss, counts, tokens = binding.balance_loss(z, ids)
    assert float(loss) == 1.0 and bool((counts == 16).all()) and int(tokens) == 64
    dz = binding.balance_loss_backward(torch.ones((), device="cuda"), z, counts, tokens)
    assert bool((dz == 0).all())  # nothing to even out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [40, 700])
def test_balance_special_logits(T, dtype):
    """Masked experts (-infinity and the type's lowest value), rows without any expert, and whatever a
    token that does not count holds."""
    torch = _torch()
    E = 100
    z, ids, _ = case(T, E, E + 1, dtype, "no", T)
    z[:, 5] = float("-inf")
    z[:, 6] = torch.finfo(z.dtype).min
    z[3, :E] = float("-inf")
    z[4, :E] = torch.finfo(z.dtype).min
    z[:, E] = float("nan")  # not an expert's column
    mask = torch.ones((T,), dtype=torch.uint8, device="cuda")
    mask[7::9] = 0
    mask[2] = 200
    z[7::9] = float("nan")
    ids[7::9] = -3
    clean = z.clone()
    clean[7::9] = 0
    check(clean, ids, E, mask)
    a, b = binding.balance_loss(z, ids, E, mask), binding.balance_loss(clean, ids, E, mask)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    d = torch.ones((), device="cuda")
    assert torch.equal(binding.balance_loss_backward(d, z, a[1], a[2], mask),
                       binding.balance_loss_backward(d, clean, a[1], a[2], mask))
    z[1, 9] = float("nan")
    assert bool(binding.balance_loss(z, ids, E, mask)[0].isnan())
    dz = binding.balance_loss_backward(d, z, a[1], a[2], mask)
    assert bool(dz[1, :E].isnan().all()) and not bool(dz[2:].isnan().any())
    z[1, 9] = float("inf")
    assert bool(binding.balance_loss(z, ids, E, mask)[0].isnan())


def test_balance_against_differences():
    """The gradient against central differences of the 64-bit loss (counts held)."""
    torch = _torch()
    T, E = 24, 16
    z, ids, mask = case(T, E, E + 1, "f32", "some", 5)
    _, c, tokens = binding.balance_loss(z, ids, E, mask)
    dz = binding.balance_loss_backward(torch.ones((), device="cuda"), z, c, tokens, mask).double()
    _, _, n, f = plain(z, ids, E, mask)

    def loss(v):
        return E * float((f * plain(v, ids, E, mask)[0].sum(0)).sum()) / n

    h = 1e-5
    g = gen(6)
    for _ in range(20):
        d = torch.randn((T, E + 1), generator=g, device="cuda", dtype=torch.float64)
        slope = (loss(z.double() + h * d) - loss(z.double() - h * d)) / (2 * h)
        # differences: h^2 / 6 times a third derivative of order 1; the gradient: fp32
        assert abs(float((dz * d).sum()) - slope) < 1e-6


def test_balance_of_a_hot_expert_and_large_batch():
    """Every token on the same eight of 256 experts; a million tokens."""
    torch = _torch()
    T, E = 1 << 20, 256
    g = gen(8)
    z = torch.randn((T, E), generator=g, device="cuda").to(torch.bfloat16)
    z[:, :8] += 6
    ids = torch.arange(8, dtype=torch.int32, device="cuda").expand(T, 8).contiguous()
    loss, counts, tokens = binding.balance_loss(z, ids)
    assert counts[:8].tolist() == [T] * 8 and int(counts[8:].sum()) == 0 and int(tokens) == T
    mean = sum(torch.softmax(z[i:i + 65536].double(), 1).sum(0) for i in range(0, T, 65536)) / T
    want = E / 8 * float(mean[:8].sum())
    assert abs(float(loss) - want) <= want * ((2.5 * 20 + 30) * U + 140 * U)
    dz = binding.balance_loss_backward(torch.ones((), device="cuda"), z, counts, tokens)
    p = torch.softmax(z[-1000:].double(), 1)
    f = counts.double() / (8 * T)
    want = E / T * p * (f - (p * f).sum(1, keepdim=True))
    err = (dz[-1000:].double() - want).abs()
    assert bool((err <= 2.0 ** -8 * 1.01 * want.abs() + 1e-5 * E / T * p).all())


def test_balance_of_ranks_summed():
    """Counts and tokens summed over two shares of the tokens give the gradient of the whole."""
    torch = _torch()
    z, ids, _ = case(1000, 64, 65, "f32", "no", 9)
    _, c, n = binding.balance_loss(z, ids, 64)
    parts = [binding.balance_loss(z[a:b], ids[a:b], 64) for a, b in ((0, 300), (300, 1000))]
    assert torch.equal(parts[0][1] + parts[1][1], c) and int(parts[0][2] + parts[1][2]) == int(n)
    d = torch.ones((), device="cuda")
    whole = binding.balance_loss_backward(d, z, c, n)
    share = binding.balance_loss_backward(d, z[:300], c, n)
    assert torch.equal(whole[:300], share)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,E", [(0, 8), (1, 8), (3, 9), (4, 256), (31, 64), (33, 255), (257, 60), (4097, 256),
                                 (20000, 128)])
def test_route_backward(T, E, gated):
    torch = _torch()
    g = gen(T + E)
    z = torch.randn((T, E), generator=g, device="cuda")
    top, ids = z.topk(8, dim=1)
    w, ids = torch.softmax(top, 1), ids.to(torch.int32)
    dw = torch.randn((T, 8), generator=g, device="cuda")
    gate = torch.sigmoid(torch.randn((T,), generator=g, device="cuda")) if gated else None
    dgate = torch.randn((T,), generator=g, device="cuda") if gated else None
    out = torch.full((T, E + gated), 7.5, device="cuda")
    got = binding.route_backward(dw, w, ids, E, dgate, gate, dlogits=out)
    assert got is out
    w64, dw64 = w.double(), dw.double()
    v = w64 * (dw64 - (w64 * dw64).sum(1, keepdim=True))
    want = torch.zeros((T, E + gated), dtype=torch.float64, device="cuda")
    want.scatter_add_(1, ids.long(), v)
    # products, three additions of the dot, a difference, a product
    size = torch.zeros_like(want).scatter_add_(1, ids.long(), w64 * (dw64.abs() + (w64 * dw64).abs().sum(1, keepdim=True)))
    bound = 8 * U * size + 2.0 ** -140
    if gated:
        g64 = gate.double()
        want[:, E] = g64 * (1 - g64) * dgate.double()
        bound[:, E] = 4 * U * want[:, E].abs() + 2.0 ** -140
    assert bool(((got.double() - want).abs() <= bound).all())


def test_route_backward_repeated_and_dropped():
    """An id that a token names more than once takes the sum of its ranks; ids outside are dropped."""
    torch = _torch()
    T, E = 40, 16
    g = gen(3)
    ids = torch.randint(-2, E + 2, (T, 8), generator=g, device="cuda", dtype=torch.int32)
    ids[0] = 5
    ids[1] = -1
    # whole eighths: every product and sum is exact
    w = torch.full((T, 8), 0.125, device="cuda")
    dw = torch.randint(-8, 9, (T, 8), generator=g, device="cuda").float() * 8
    got = binding.route_backward(dw, w, ids, E)
    v = w * (dw - (w * dw).sum(1, keepdim=True))
    want = torch.zeros((T, E), device="cuda")
    for t in range(T):
        for k in range(8):
            if 0 <= int(ids[t, k]) < E:
                want[t, int(ids[t, k])] += v[t, k]
    assert torch.equal(got, want)


def layer():
    w = inputs.BY_NAME["tiny_fp32_t4"]
    m, t = binding.layer_from_numpy(inputs.make_layer(w), max_tokens=256)
    return m, t, w


def test_route_is_recorded():
    torch = _torch()
    m, _, wl = layer()
    E, T = wl.num_experts, 37
    z = torch.randn((T, m.rows), generator=gen(11), device="cuda", requires_grad=True)
    plain_out = m.route(logits=z.detach())
    zz, ids, w, g = m.route(logits=z)
    for a, b in zip(plain_out, (zz, ids, w, g)):
        assert torch.equal(a, b)
    assert w.requires_grad and g.requires_grad and not zz.requires_grad and not ids.requires_grad
    cw, cg = torch.randn_like(w), torch.randn_like(g)
    ((w * cw).sum() + (g * cg).sum()).backward()
    z64 = z.detach().double().requires_grad_()
    w64 = torch.softmax(z64.gather(1, ids.long()), 1)
    ((w64 * cw.double()).sum() + (torch.sigmoid(z64[:, E]) * cg.double()).sum()).backward()
    # w itself is within 1e-6 of the exact one (the layer's own bound)
    assert float((z.grad.double() - z64.grad).abs().max()) < 2e-5
    z.grad = None
    m.route(logits=z, T=20, want_logits=False)[2].square().sum().backward()
    assert bool((z.grad[20:] == 0).all()) and bool((z.grad[:20] != 0).any())
    z.grad = None
    m.route(logits=z)[3].sum().backward()  # the gate only
    assert bool((z.grad[:, :E] == 0).all())
    with torch.no_grad():
        assert not m.route(logits=z)[2].requires_grad
    with pytest.raises(ValueError):
        m.route(logits=z[:, :-1])
    # no second derivative
    s = m.route(logits=z)[2].square().sum()
    (d,) = torch.autograd.grad(s, z, create_graph=True)
    with pytest.raises(RuntimeError):
        d.sum().backward()
    m.close()


def test_balance_is_recorded():
    torch = _torch()
    z, ids, mask = case(300, 64, 65, "f32", "some", 12)
    z.requires_grad_()
    loss, counts, tokens = binding.balance_loss(z, ids, 64, mask)
    assert loss.requires_grad and not counts.requires_grad
    (3 * loss).backward()
    want = binding.balance_loss_backward(torch.tensor(3.0, device="cuda"), z.detach(), counts, tokens, mask)
    assert torch.equal(z.grad, want)
    assert not binding.balance_loss(z.detach(), ids, 64, mask)[0].requires_grad


def test_streams():
    torch = _torch()
    z, ids, mask = case(3000, 256, 257, "f32", "some", 13)
    first = binding.balance_loss(z, ids, 256, mask)
    d = torch.ones((), device="cuda")
    dz = binding.balance_loss_backward(d, z, first[1], first[2], mask)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        other = binding.balance_loss(z, ids, 256, mask, stream=side)
        dz2 = binding.balance_loss_backward(d, z, other[1], other[2], mask, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, other)) and torch.equal(dz, dz2)


@pytest.mark.parametrize("T", [100, 5000])
def test_graph_replays(T):
    """Loss and gradients captured together, replayed over new logits and ids with eager calls between."""
    torch = _torch()
    E = 128
    z, ids, mask = case(T, E, E + 1, "f32", "some", 14)
    w = torch.rand((T, 8), device="cuda")
    dw = torch.rand((T, 8), device="cuda")
    gate = torch.rand((T,), device="cuda")
    d = torch.ones((), device="cuda")

    def step():
        loss, c, n = binding.balance_loss(z, ids, E, mask)
        return loss, c, n, binding.balance_loss_backward(d, z, c, n, mask), binding.route_backward(dw, w, ids, E, gate, gate)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(5):
        z2, ids2, _ = case(T, E, E + 1, "f32", "no", 20 + i)
        z.copy_(z2)
        ids.copy_(ids2)
        dw.copy_(torch.rand((T, 8), device="cuda"))
        graph.replay()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), i


def test_router_over_4_bit_experts():
    """The operators as they are used together: a router tuned over frozen 4-bit experts. One step's
    gradient of the router's weights against the same step in 64 bits."""
    torch = _torch()
    m, _, wl = layer()
    E, T, H, I = wl.num_experts, 96, 64, 64
    g = gen(30)
    x = torch.randn((T, H), generator=g, device="cuda")
    wr = (torch.randn((m.rows, H), generator=g, device="cuda") / 8).requires_grad_()

    def experts(M, K):
        w = torch.randint(0, 256, (E, M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        return w, 0.02 + 0.01 * torch.rand((E, K // 32, M), generator=g, device="cuda")

    gu, gus = experts(2 * I, H)
    dn, dns = experts(H, I)
    shared = torch.randn((T, H), generator=g, device="cuda")
    target = torch.randn((T, H), generator=g, device="cuda")
    z = x @ wr.t()
    _, ids, w, gate = m.route(logits=z)
    _, offsets, _, rows = m.bucket_rows(ids)
    xs = binding.permute(x, rows)
    h = binding.matmul_w4(xs, gu, gus, offsets=offsets, swiglu=True, dtype=torch.float32)
    ys = binding.matmul_w4(h, dn, dns, offsets=offsets, dtype=torch.float32)
    y = binding.unpermute(ys, rows, w, shared=shared, gate=gate)
    balance, counts, tokens = binding.balance_loss(z, ids, E)
    assert int(counts.sum()) == 8 * T and torch.equal(counts, (offsets[1:] - offsets[:-1]))
    ((y - target).square().mean() + 0.1 * balance).backward()

    def full(w, s):
        c = torch.stack([w & 15, w >> 4], -1).reshape(*w.shape[:2], -1).double() - 8
        return c * s.double().transpose(1, 2).repeat_interleave(32, dim=2)

    wr64 = wr.detach().double().requires_grad_()
    z64 = x.double() @ wr64.t()
    w64 = torch.softmax(z64.gather(1, ids.long()), 1)
    y64 = torch.sigmoid(z64[:, E:]) * shared.double()
    gu64, dn64 = full(gu, gus), full(dn, dns)
    for e in range(E):
        t, k = (ids == e).nonzero(as_tuple=True)
        a = x[t].double() @ gu64[e].t()
        a = a[:, :I] * torch.sigmoid(a[:, :I]) * a[:, I:]
        y64 = y64.index_add(0, t, w64[t, k][:, None] * (a @ dn64[e].t()))
    f = counts.double() / (8 * T)
    b64 = E * (f * torch.softmax(z64[:, :E], 1).mean(0)).sum()
    ((y64 - target.double()).square().mean() + 0.1 * b64).backward()
    assert float((y.detach().double() - y64.detach()).norm() / y64.detach().norm()) < 2e-6
    # w within 1e-6 of the exact one (the layer's own bound) over values of order 0.1 and above
    assert float((wr.grad.double() - wr64.grad).norm() / wr64.grad.norm()) < 2e-5
    m.close()
