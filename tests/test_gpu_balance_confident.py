"""The balance loss's gradient for tokens that are sure of an expert, against 64 bits.

u = 2^-24, A the largest difference of a row's logits. A probability's relative error is at most REL =
(2.5 A + 30) u, that of a row's sums 22 u more (16 + 4 additions, their products). With d_e the experts' shares (about the
even one) and D = sum p d their mean, the gradient's terms are p_e (d_e - D). A mean that is subtracted twice, the
second time as the mean of what the first left over, is off in the first by at most (REL + 22u) sum p |d|, which the
second takes off again up to that factor once more, and in the second by the same factor of sum p |d - D|. So the error
is at most p_e e (|d_e - D| + sum p |d - D| + 2 e (|d_e| + sum p |d|)) with e = 2 REL + 30 u, and half a step of
the result's type: it goes to 0 with 1 - p of the expert that a token is sure of, where rounding D alone
would leave u |d|.
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


@pytest.mark.parametrize("counted", ["its own", "hot", "several ranks'"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,E,R", [(24, 8, 9), (200, 60, 61), (700, 256, 257), (3000, 256, 256), (333, 128, 128)])
def test_confident_tokens(T, E, R, dtype, counted):
    torch = _torch()
    g = torch.Generator(device="cuda")
    g.manual_seed(T + E)
    z = torch.randn((T, R), generator=g, device="cuda") * 0.5
    # 1 - p from about 1 to 1e-13, on an expert of the token's own
    sure = torch.randint(0, E, (T,), generator=g, device="cuda")
    up = torch.rand((T,), generator=g, device="cuda") * 36
    z[torch.arange(T, device="cuda"), sure] += up
    z = z.to(getattr(torch, dtype))
    ids = z[:, :E].topk(8, dim=1).indices.to(torch.int32)
    if counted == "hot":
        ids[:, 0] = E // 2
    mask = torch.rand((T,), generator=g, device="cuda") < 0.8
    _, counts, tokens = binding.balance_loss(z, ids, E, mask)
    if counted == "several ranks'":  # counts far past 2^24
        counts = (counts.long() * 300007).int()
        counts[0] += 8
        tokens = (tokens.long() * 300007 + 1).int()
    dloss = torch.tensor(0.37, device="cuda")
    got = binding.balance_loss_backward(dloss, z, counts, tokens, mask).double()

    n = int(tokens)
    p = torch.softmax(z[:, :E].double(), 1)
    # whole numbers, exact in 64 bits; the even share is the origin, which the gradient does not depend on
    d = counts.double() - 8.0 * n / E
    k = float(dloss.double()) * E / (8.0 * n * n)
    far = (d[None, :] - (p * d).sum(1, keepdim=True))
    # for the expert that a token is sure of: d_j - sum p d = sum over the others of p (d_j - d)
    top = p.argmax(1)
    gap = d[top][:, None] - d[None, :]
    others = p.clone()
    others[torch.arange(T, device="cuda"), top] = 0
    far[torch.arange(T, device="cuda"), top] = (others * gap).sum(1)
    want = k * p * far * mask[:, None]

    A = float((z[:, :E].amax(1) - z[:, :E].amin(1)).max())
    e = 2 * (2.5 * A + 30) * U + 30 * U
    bound = k * p * e * (far.abs() + (p * far.abs()).sum(1, keepdim=True) +
                         2 * e * (d.abs()[None, :] + (p * d.abs()).sum(1, keepdim=True)))
    # 64 bits' own: p's roundings
    bound = bound * 1.01 + torch.finfo(z.dtype).eps / 2 * want.abs() + 2.0 ** -120
    if counted == "several ranks'":  # each share is one fp32 number: half a step of it
        bound = bound + k * p * U * 1.01 * (d.abs()[None, :] + (p * d.abs()).sum(1, keepdim=True))
    bad = (got[:, :E] - want).abs() > bound
    assert not bool(bad.any()), (int(bad.sum()), float(((got[:, :E] - want).abs() / bound).max()))
    assert bool((got[:, E:] == 0).all()) and bool((got[~mask] == 0).all())


def test_the_expert_a_token_is_sure_of():
    """Two experts with probabilities 1 - q and nearly q, counts 16 and 0 apart: q d / (1 - q) is the whole of it."""
    torch = _torch()
    E, T = 16, 60
    z = torch.full((T, E), -60.0, device="cuda")
    x = torch.linspace(0.0, 24.0, T, device="cuda")
    z[:, 3], z[:, 9] = x, 0.0
    counts = torch.full((E,), 30, dtype=torch.int32, device="cuda")
    counts[3], counts[9] = 38, 22
    tokens = torch.tensor(60, dtype=torch.int32, device="cuda")
    got = binding.balance_loss_backward(torch.ones((), device="cuda"), z, counts, tokens).double()
    q = torch.sigmoid(-x.double())
    want = E / (8.0 * 60 * 60) * q * (1 - q) * 16
    # relative: two probabilities and the sums, and 1 - q of the nearest fp32 numbers of p
    rel = 4 * (2.5 * 84 + 30) * U
    assert bool(((got[:, 3] - want).abs() <= rel * want + 1e-12 * rel).all()), ((got[:, 3] - want) / want).abs().max()
    assert bool(((got[:, 9] + want).abs() <= rel * want + 1e-12 * rel).all())
