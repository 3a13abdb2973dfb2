"""Cross entropy gradients at labels, up to probabilities of 1 - 1e-6, against their entries in 64
bits for the given lse (tests/training_labels.py derives the bounds)."""
import pytest
import torch

import embedding_table_gather_amd as etg
from tests import training_labels as tl
from tests.gpu_util import note

pytestmark = pytest.mark.gpu
CODES = {torch.float32: etg.F32, torch.bfloat16: etg.BF16, torch.float16: etg.F16}


def _check(got, want, bound, what):
    off = (got.double().cpu() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float((off / bound).max()):.3g} of the bound"


@pytest.mark.parametrize("zloss", [False, True])
@pytest.mark.parametrize("case", tl.CASES, ids=str)
def test_confident_labels(case, zloss):
    note(f"labels {case}, zloss {zloss}")
    dtype, n, V, d = tl.TYPES[case[0]], *case[1:]
    E, x, labels, Y = tl.make(n, V, d, dtype)
    g, h = tl.upstream(n, dtype)
    h = h if zloss else None
    t = etg.Table(E.cuda(), CODES[dtype], V, d)
    xd, yd = x.cuda(), labels.cuda()
    _, lse = t.cross_entropy(xd, yd)
    dx, dE = t.cross_entropy_grad(xd, yd, lse, g.cuda(), None if h is None else h.cuda())
    torch.cuda.synchronize()
    entry, bound = tl.entries(E, x, labels, lse.cpu(), g, h)
    wx, tx, wE, tE = tl.shown(E, x, labels, Y, entry, bound, n <= 128)
    got_x, got_E = tl.pick(dx.cpu(), dE.cpu(), x, Y)
    has = labels >= 0
    _check(got_x[has], wx[has], tx[has], "residual gradient")
    _check(got_E, wE, tE, "table gradient")


@pytest.mark.parametrize("dtype", sorted(tl.TYPES))
def test_unaligned_rows_have_the_same_entries(dtype):
    T = tl.TYPES[dtype]
    n, V, d = 40, 20011, 136
    note(f"labels, strided rows {dtype}")
    E, x, labels, Y = tl.make(n, V, d, T, seed=3)
    g, h = tl.upstream(n, T)
    t = etg.Table(E.cuda(), CODES[T], V, d)
    wide = torch.full((n, d + 3), float("nan"), dtype=T, device="cuda")
    wide[:, :d] = x.cuda()
    _, lse = t.cross_entropy(x.cuda(), labels.cuda())
    a = t.cross_entropy_grad(x.cuda(), labels.cuda(), lse, g.cuda(), h.cuda())
    b = t.cross_entropy_grad(wide[:, :d], labels.cuda(), lse, g.cuda(), h.cuda())
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("case", tl.CANCELLING, ids=str)
def test_loss_of_cancelling_label_logits(case):
    note(f"cancelling {case}")
    dtype, n, V, d = tl.TYPES[case[0]], *case[1:]
    E, x, labels = tl.make_cancelling(n, V, d, dtype)
    t = etg.Table(E.cuda(), CODES[dtype], V, d)
    loss, lse = t.cross_entropy(x.cuda(), labels.cuda())
    torch.cuda.synchronize()
    want, want_lse, tol, tol_lse = tl.loss_of(E, x, labels)
    _check(lse, want_lse, tol_lse, "lse")
    _check(loss, want, tol, "loss")


@pytest.mark.parametrize("dtype", sorted(tl.TYPES))
@pytest.mark.parametrize("n,V,d", [(1, 1, 8), (5, 1, 64), (40, 700, 128), (100, 20011, 264), (300, 3001, 1024)])
def test_losses_of_sure_labels_are_never_negative(dtype, n, V, d):
    # probabilities that round to 1, sums that an f32 accumulator gets wrong by more than 1 - p
    note(f"sure labels {dtype} {n} x {V} x {d}")
    T = tl.TYPES[dtype]
    gen = torch.Generator().manual_seed(n + V)
    E = torch.randn((V, d), generator=gen).to(T)
    x = torch.randn((n, d), generator=gen)
    at = torch.randint(V, (n,), generator=gen, dtype=torch.int32)
    target = E[at.long()].float()
    x += target * (60 / target.square().sum(1, keepdim=True))
    x = x.to(T)
    t = etg.Table(E.cuda(), CODES[T], V, d)
    loss, lse = t.cross_entropy(x.cuda(), at.cuda())
    torch.cuda.synchronize()
    L = x.double() @ E.double().t().contiguous()
    want = torch.logsumexp(L, 1)
    assert (loss >= 0).all()
    if V == 1:
        assert (loss <= 1e-9).all()
    dL = d * 2.0 ** -22 * (x.double().abs() @ E.double().abs().t().contiguous()).max(1).values
    _check(lse.cpu(), want, dL + 1e-5 + want.abs() * 2.0 ** -24, "lse")
    _check(loss.cpu(), want - L.gather(1, at.long()[:, None])[:, 0], dL + 1e-5, "loss")
