"""The recorded balance loss and the counts it hands out: they are the caller's, to be summed over ranks in
place, and the gradient stays that of the loss that was computed. A collective writes into a tensor
without raising its version counter, so that autograd cannot see it."""

import pytest

from sparse_moe_routing_amd import binding


def plain_loss(logits, ids, num_experts, mask=None):
    """(loss, counts, tokens) on any device, from the definition."""
    import torch
    on = torch.ones(len(ids), dtype=torch.bool, device=ids.device) if mask is None else mask
    counts = torch.bincount(ids[on].reshape(-1).long(), minlength=num_experts).int()
    n = on.sum().int()
    p = torch.softmax(logits[on][:, :num_experts], 1).sum(0)
    return (counts * p).sum() * num_experts / (8.0 * n * n), counts, n


def plain_grad(dloss, logits, counts, tokens, mask=None):
    import torch
    E = counts.numel()
    p = torch.softmax(logits[:, :E], 1)
    f = counts / (8.0 * tokens)
    d = p * (f - (p * f).sum(1, keepdim=True)) * (dloss * E / tokens)
    if mask is not None:
        d = d * mask[:, None]
    out = torch.zeros_like(logits)
    out[:, :E] = d
    return out


def inputs(device="cpu", seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((40, 17), generator=g)
    ids = z[:, :16].topk(8, dim=1).indices.int()
    mask = torch.rand((40,), generator=g) < 0.7
    return z.to(device), ids.to(device), mask.to(device)


@pytest.fixture
def plain(monkeypatch):
    """The operators' plain forms in the library's place, on CPU tensors."""
    loss = binding.balance_loss

    def run(logits, ids, num_experts=None, mask=None, stream=None):
        import torch
        if logits.requires_grad and torch.is_grad_enabled():
            return loss(logits, ids, num_experts, mask)
        return plain_loss(logits, ids, num_experts, mask)

    monkeypatch.setattr(binding, "_switched", lambda device, stream: None)
    monkeypatch.setattr(binding, "balance_loss", run)
    monkeypatch.setattr(binding, "balance_loss_backward", plain_grad)


def written(t, by):
    t.data += by  # as a collective writes: the version counter stays


def test_counts_written_before_the_backward_pass(plain):
    import torch
    z, ids, mask = inputs()
    _, c, n = plain_loss(z, ids, 16, mask)
    want = plain_grad(torch.tensor(2.0), z, c, n, mask)
    z.requires_grad_()
    for change in ((5, 0), (0, 7), (5, 7), (-3, 0)):
        loss, counts, tokens = binding.balance_loss(z, ids, 16, mask)
        assert torch.equal(counts, c) and int(tokens) == int(n) and tokens.shape == ()
        assert not counts.requires_grad and not tokens.requires_grad
        written(counts, change[0])
        written(tokens, change[1])
        version = counts._version
        z.grad = None
        (2 * loss).backward()
        assert version == 0 and torch.equal(z.grad, want), change
        assert torch.equal(counts, c + change[0])  # and the caller's stay the caller's


def test_two_backward_passes_see_the_same_counts(plain):
    import torch
    z, ids, mask = inputs(seed=1)
    z.requires_grad_()
    loss, counts, tokens = binding.balance_loss(z, ids, 16, mask)
    (first,) = torch.autograd.grad(loss, z, retain_graph=True)
    written(counts, 9)
    (second,) = torch.autograd.grad(loss, z)
    assert torch.equal(first, second)


def _rank(rank, port, out):
    import torch
    import torch.distributed as dist
    dist.init_process_group("gloo", init_method=f"tcp://127.0.0.1:{port}", rank=rank, world_size=2)
    loss = binding.balance_loss
    binding._switched = lambda device, stream: None
    binding.balance_loss = lambda *a, **k: loss(*a, **k) if a[0].requires_grad and torch.is_grad_enabled() else plain_loss(*a, **k)
    binding.balance_loss_backward = plain_grad
    z, ids, mask = inputs(seed=2 + rank)
    z.requires_grad_()
    value, counts, tokens = binding.balance_loss(z, ids, 16, mask)
    want = plain_grad(torch.tensor(1.0), z.detach(), counts.clone(), tokens.clone(), mask)
    mine = counts.clone()
    dist.all_reduce(counts)  # the load over all ranks, for statistics
    value.backward()
    out.put((rank, bool(torch.equal(z.grad, want)), int(counts.sum() - mine.sum())))
    dist.barrier()
    dist.destroy_process_group()


def test_counts_summed_over_two_ranks():
    import socket
    import torch.multiprocessing as mp
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    out = ctx.Queue()
    ranks = [ctx.Process(target=_rank, args=(r, port, out)) for r in range(2)]
    for p in ranks:
        p.start()
    got = [out.get(timeout=100) for _ in ranks]
    for p in ranks:
        p.join(timeout=60)
        assert p.exitcode == 0
    for rank, same, others in sorted(got):
        assert same and others > 0, rank


def test_calls_of_a_recorded_loss(monkeypatch):
    """One call of the library forwards and one backwards, over the caller's logits and mask and counts that
    nobody else holds."""
    import torch
    from test_w4_router_refusals import good
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
    _, a = good("cpu")["balance_loss"]
    z = a["logits"].requires_grad_()
    loss, counts, tokens = binding.balance_loss(**a)
    assert loss.requires_grad and not counts.requires_grad and not tokens.requires_grad
    loss.backward()
    assert [name for name, _ in seen] == ["moe_balance_loss", "moe_balance_loss_backward"]
    _, pz, pc, pt, pm = seen[1][1][:5]
    assert (pz, pm) == (z.data_ptr(), a["mask"].data_ptr())
    assert pc != counts.data_ptr() and pt != tokens.data_ptr()
    assert z.grad.shape == z.shape
    with torch.no_grad():
        assert not binding.balance_loss(**a)[0].requires_grad


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("change", [(5, 0), (0, 7), (5, 7)])
def test_counts_written_on_the_device(change, dtype):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    z, ids, mask = inputs("cuda")
    z = z.to(getattr(torch, dtype))
    _, c, n = binding.balance_loss(z, ids, 16, mask)
    want = binding.balance_loss_backward(torch.tensor(2.0, device="cuda"), z, c, n, mask)
    z.requires_grad_()
    loss, counts, tokens = binding.balance_loss(z, ids, 16, mask)
    assert torch.equal(counts, c) and int(tokens) == int(n)
    written(counts, change[0])
    written(tokens, change[1])
    (2 * loss).backward()
    assert torch.equal(z.grad, want)


@pytest.mark.gpu
def test_recorded_loss_in_a_graph():
    """Loss and its recorded gradient in one captured graph, replayed over other logits while the counts of the
    replay before are written into. The leaf of the graph is its own: made inside the capture."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    z, ids, mask = inputs("cuda", 3)
    dloss = torch.tensor(0.5, device="cuda")

    def step():
        leaf = z.detach().requires_grad_()
        loss, counts, tokens = binding.balance_loss(leaf, ids, 16, mask)
        counts.add_(1)  # seen by nobody else
        (d,) = torch.autograd.grad(loss, leaf, dloss)
        return loss.detach(), counts, tokens, d

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        z2, ids2, _ = inputs("cuda", 10 + i)
        z.copy_(z2)
        ids.copy_(ids2)
        graph.replay()
        torch.cuda.synchronize()
        loss, c, n = binding.balance_loss(z, ids, 16, mask)
        want = (loss, c + 1, n, binding.balance_loss_backward(dloss, z, c, n, mask))
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        out[1].data.add_(100)
