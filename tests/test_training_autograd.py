"""Autograd around the training operators: the warning on the host, the documented function on the GPU."""
import warnings

import pytest
import torch

import embedding_table_gather_amd as etg


def _host_table():
    t = etg.Table.__new__(etg.Table)  # a table's arguments without a device: every call is refused later on
    t.dtype, t.vocab, t.hidden, t.device = etg.BF16, 4, 8, torch.device("cpu")
    return t


def test_a_residual_that_requires_grad_is_warned_of():
    t, y = _host_table(), torch.zeros(3, dtype=torch.int32)
    x = torch.zeros((3, 8), dtype=torch.bfloat16, requires_grad=True)
    with pytest.warns(UserWarning, match="requires grad"), pytest.raises(ValueError):
        t.cross_entropy(x, y)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with torch.no_grad(), pytest.raises(ValueError):
            t.cross_entropy(x, y)
        with pytest.raises(ValueError):
            t.cross_entropy(x.detach(), y)


class TiedLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, table, labels, t):
        loss, lse = t.cross_entropy(x, labels)
        ctx.save_for_backward(x, labels, lse)
        ctx.t = t
        return loss

    @staticmethod
    def backward(ctx, g):
        x, labels, lse = ctx.saved_tensors
        dx, dt = ctx.t.cross_entropy_grad(x, labels, lse, g.contiguous())
        return dx, dt, None, None


@pytest.mark.gpu
@pytest.mark.parametrize("reduce", ["mean", "sum", "weighted"])
def test_a_function_with_a_backward_pass_of_its_own(reduce):
    from tests import training_oracle as to
    n, V, d = 40, 700, 64
    gen = torch.Generator().manual_seed(5)
    E = (torch.randn((V, d), generator=gen) * 0.1).bfloat16().cuda().requires_grad_()
    x = torch.randn((n, d), generator=gen).bfloat16().cuda().requires_grad_()
    labels = torch.randint(-1, V, (n,), generator=gen, dtype=torch.int32).cuda()
    w = torch.rand(n, generator=gen).cuda()
    t = etg.Table(E.detach(), etg.BF16, V, d)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        loss = TiedLoss.apply(x, E, labels, t)
    {"mean": loss.mean(), "sum": loss.sum(), "weighted": (loss * w).sum()}[reduce].backward()
    torch.cuda.synchronize()
    g = {"mean": torch.full((n,), 1 / n), "sum": torch.ones(n), "weighted": w.cpu()}[reduce]
    with torch.no_grad():
        _, lse = t.cross_entropy(x, labels)
    wx, wE, tx, tE = to.grads(x.detach().cpu(), E.detach().cpu(), labels.cpu(), lse.cpu(), g)
    to.check(x.grad, wx, tx, "residual gradient")
    to.check(E.grad, wE, tE, "table gradient")
