"""Arguments of the router's training entry points as autograd hands them out,
and refusals of the binding."""
import pytest
import torch

from mixture_experts_layer_up_amd import binding
from tests._gpu import announce

pytestmark = pytest.mark.gpu


def _call(d_loss, T=24, E=16, k=2):
    sh = binding.Shape(T, 64, 32, E, k, 0, E, 0, 0, 0, 1.0, 0, 0)
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn((T, E), generator=g, device="cuda")
    ids = x.topk(k).indices.int()
    bal = binding.balance_loss(sh, x, ids)
    return binding.route_backward(sh, x, balance=bal, d_loss=d_loss)


def test_gradient_of_the_loss_without_dimensions():
    """A scalar loss has a gradient without dimensions: the same bits as [1]."""
    announce("d_loss without dimensions")
    want = _call(torch.full((1,), 0.7, device="cuda"))
    assert torch.equal(_call(torch.tensor(0.7, device="cuda")), want)


def test_autograd_function_around_the_loss():
    """The loss inside a torch graph: scaled, summed with another, backward."""
    T, E, k = 40, 8, 2
    sh = binding.Shape(T, 64, 32, E, k, 0, E, 0, 0, 0, 1.0, 0, 0)

    class Balance(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, ids):
            ctx.bal = binding.balance_loss(sh, x, ids)
            ctx.save_for_backward(x)
            return ctx.bal["loss"].view(())

        @staticmethod
        def backward(ctx, d_loss):
            return binding.route_backward(sh, ctx.saved_tensors[0], balance=ctx.bal, d_loss=d_loss), None

    announce("balance loss in a graph")
    x = torch.randn((T, E), device="cuda", generator=torch.Generator("cuda").manual_seed(4), requires_grad=True)
    ids = x.detach().topk(k).indices.int()
    (0.5 * Balance.apply(x, ids) + (x * x).sum()).backward()
    z = x.detach().double().requires_grad_()
    n = torch.bincount(ids.view(-1).long(), minlength=E).double()
    (0.5 * E / (k * T) * (n * z.softmax(1).mean(0)).sum() + (z * z).sum()).backward()
    # (2 E + 2 k + 40 + 2 span) roundings of the loss's terms (< 1), one each of 2 x and of the sum
    assert ((x.grad - z.grad).abs() <= 2.0 ** -24 * (80 + 4 * z.grad.abs())).all()


@pytest.mark.parametrize("bad,what", [
    (torch.ones((1, 1)), "d_loss has shape"), (torch.ones(2), "d_loss has shape"),
    (torch.ones(1, dtype=torch.float64), "dtype"), (torch.tensor(1.0, dtype=torch.bfloat16), "dtype")])
def test_bad_gradients_of_the_loss(bad, what):
    with pytest.raises(binding.MoELoRAError, match=what):
        _call(bad.cuda())
    with pytest.raises(binding.MoELoRAError, match="one GPU"):
        _call(torch.tensor(1.0))
