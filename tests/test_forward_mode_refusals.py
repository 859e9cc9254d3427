"""Forward-mode derivatives: the operators that autograd records have none, and neither has the 4-bit
product. An operand that carries a tangent is refused before the library is called, where the tangent would
be lost; without one (a primal, a detached operand) calls go through."""
import pytest

from sparse_moe_routing_amd import binding
import test_operators_binding as rows_binding
import test_w4_router_refusals as w4_binding

# the operands that a derivative would be with respect to
CASES = [("permute", "x"), ("unpermute", "ys"), ("unpermute", "w"), ("unpermute", "shared"), ("unpermute", "gate"),
         ("matmul_w4", "x"), ("matmul_w4", "scale"), ("balance_loss", "logits")]


def good(op, device):
    table = w4_binding if op in w4_binding.OPERATORS else rows_binding
    return table.good(device)[op]


calls = w4_binding.calls  # the library and the device lookup stood in for


@pytest.fixture
def dual():
    import torch.autograd.forward_ad as forward
    with forward.dual_level():
        yield forward


@pytest.mark.parametrize("no_grad", [False, True])
@pytest.mark.parametrize("op,arg", CASES)
def test_tangent_is_refused(calls, dual, op, arg, no_grad):
    import torch
    f, operands = good(op, "cpu")
    plain = operands[arg]
    operands[arg] = dual.make_dual(plain, torch.ones_like(plain))
    with pytest.raises(ValueError, match="forward-mode"):
        with torch.set_grad_enabled(not no_grad):
            f(**operands)
    assert calls == []
    operands[arg] = dual.unpack_dual(operands[arg]).primal
    f(**operands)
    operands[arg] = dual.make_dual(plain, torch.ones_like(plain)).detach()
    f(**operands)
    assert [name for name, _ in calls] == ["moe_" + op] * 2


@pytest.mark.parametrize("op,arg", [c for c in CASES if c[0] != "matmul_w4"])
def test_tangent_beside_a_recorded_gradient_is_refused(calls, dual, op, arg):
    import torch
    f, operands = good(op, "cpu")
    operands = {k: v for k, v in operands.items() if k not in ("xs", "y")}
    operands[arg] = dual.make_dual(operands[arg].requires_grad_(), torch.ones_like(operands[arg]))
    with pytest.raises(ValueError, match="forward-mode"):
        f(**operands)
    assert calls == []


@pytest.mark.parametrize("no_grad", [False, True])
def test_tangent_of_given_logits_is_refused(calls, dual, no_grad):
    """MoeLayer.route: the logits that it ranks, recorded or not."""
    import torch
    layer = object.__new__(binding.MoeLayer)
    layer.lib, layer.ctx, layer.shared_inter, layer.num_experts, layer.rows = binding.load(), None, 0, 16, 16
    ws = torch.zeros(64, dtype=torch.uint8)
    z = torch.zeros((4, 16))
    for leaf in (z, z.clone().requires_grad_()):
        with pytest.raises(ValueError, match="forward-mode"):
            with torch.set_grad_enabled(not no_grad):
                layer.route(logits=dual.make_dual(leaf, torch.ones_like(z)), ws=ws)
    assert calls == []


@pytest.mark.gpu
def test_tangent_is_refused_on_the_device(dual):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    for op, arg in CASES:
        f, operands = good(op, "cuda")
        plain = operands[arg]
        operands[arg] = dual.make_dual(plain, torch.ones_like(plain))
        with pytest.raises(ValueError, match="forward-mode"):
            f(**operands)
        operands[arg] = plain
        f(**operands)
    torch.cuda.synchronize()
