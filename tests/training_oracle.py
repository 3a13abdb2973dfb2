"""Plain 64-bit forms of the tied table's training operators, with error bounds.

Written from the operators' definitions; they share no code with the library.  Everything is
torch in float64 on the device of its inputs.

The bounds count roundings.  A product of K terms accumulated in f32 by the matrix cores is
within K * 2^-22 * sum |a b| of the exact one (four unit roundoffs per term: the bound that
test_mfma_accumulation_gpu.py checks the matrix cores against); 16-bit operands' products are
exact in f32.  A rounding to a type is off by half a step, eps / 2 of the value, or half the
smallest subnormal.
"""
import torch

SUBNORMAL = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def rounding(x, dtype):
    return x.abs() * (torch.finfo(dtype).eps / 2) + SUBNORMAL[dtype] / 2


def logits(x, E):
    """(L, bound of its f32 accumulation)."""
    x, E = x.double(), E.double()
    return x @ E.t().contiguous(), x.shape[1] * 2.0 ** -22 * (x.abs() @ E.abs().t().contiguous())


def has_label(labels, V):
    return (labels >= 0) & (labels.long() < V)


def loss(x, E, labels):
    """(loss, lse, bound of loss, bound of lse).

    lse moves by at most the largest error of a row's logits.  exp2 of a difference d rounds
    its argument twice and its result to 1 ulp: 2^-23 (1 + |d|) each, and a term with |d| > 30
    weighs less than 2^-43; sums run over at most 64 values, six exchanges, eight waves and the
    tiles in turn (fewer than 100 additions for the sizes used here): 31 * 2^-23 + 100 * 2^-24
    < 1e-5.  The result is rounded once.
    """
    L, dL = logits(x, E)
    lse = torch.logsumexp(L, 1)
    d_lse = dL.max(1).values + 1e-5 + rounding(lse, torch.float32)
    ok = has_label(labels, E.shape[0])
    at = torch.where(ok, labels, torch.zeros_like(labels)).long()[:, None]
    target, d_target = L.gather(1, at)[:, 0], dL.gather(1, at)[:, 0]
    out = torch.where(ok, lse - target, torch.zeros_like(lse))
    d_out = torch.where(ok, dL.max(1).values + d_target + 1e-5 + rounding(out, torch.float32), torch.zeros_like(lse))
    return out, lse, d_out, d_lse


def grads(x, E, labels, lse, g, h=None, old=None):
    """(dx, dE, bound of dx, bound of dE) of the rows' type, for the given lse.

    D = (g + h) p - g [label]: p moves by its logit's error plus 31 * 2^-23 + 2^-23 < 4e-6 of
    itself for the exponential (|argument| <= 30; smaller terms are smaller still), the sum, the
    product and the difference round three times, and D to the table's type (f16 D is scaled so
    that the largest |g|, |g + h| lies in [2^13, 2^14): half a subnormal step is 2^-38 of it).
    """
    dtype = x.dtype
    V, K = E.shape
    n = x.shape[0]
    ok = has_label(labels, V)
    g = torch.where(ok, g.double(), torch.zeros(n, dtype=torch.float64, device=x.device))
    c = g if h is None else g + h.double()
    L, dL = logits(x, E)
    cp = torch.exp(L - lse.double()[:, None]) * c[:, None]
    hot = torch.zeros_like(L)
    hot[torch.arange(n, device=x.device)[ok], labels[ok].long()] = 1.0
    D = cp - hot * g[:, None]
    dD = cp.abs() * (torch.expm1(dL) + 4e-6) + 2.0 ** -23 * (cp.abs() + hot * g.abs()[:, None])
    dD = dD + D.abs() * (torch.finfo(dtype).eps / 2)
    if dtype == torch.float16:
        dD = dD + 2.0 ** -38 * torch.maximum(g.abs(), c.abs()).max()
    else:
        dD = dD + SUBNORMAL[dtype] / 2
    xd, Ed = x.double(), E.double()
    dx = D @ Ed
    e_x = dD @ Ed.abs() + (V + 64) * 2.0 ** -22 * ((D.abs() + dD) @ Ed.abs())
    dE = D.t().contiguous() @ xd
    e_E = dD.t().contiguous() @ xd.abs() + (n + 1) * 2.0 ** -22 * ((D.abs() + dD).t().contiguous() @ xd.abs())
    if old is not None:
        dE = dE + old.double()
        e_E = e_E + 2.0 ** -24 * (dE.abs() + e_E)
    return dx, dE, e_x + rounding(dx, dtype) + e_x * torch.finfo(dtype).eps, \
        e_E + rounding(dE, dtype) + e_E * torch.finfo(dtype).eps


def gather_grad(grad, ids, V, scale, dtype, old=None):
    """(out, bound): a sum of m rows rounds m times, the scale and the addition once each, the
    result to its type."""
    ok = has_label(ids, V)
    at, rows = ids[ok].long(), grad[ok].double()
    out = torch.zeros((V, grad.shape[1]), dtype=torch.float64, device=grad.device)
    mass = out.clone()
    count = torch.zeros(V, dtype=torch.float64, device=grad.device)
    out.index_add_(0, at, rows)
    mass.index_add_(0, at, rows.abs())
    count.index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    e = (count[:, None] + 1) * 2.0 ** -24 * mass * abs(scale)
    out = out * scale
    if old is not None:
        out = out + old.double()
        e = e + 2.0 ** -24 * (out.abs() + e)
    return out, e + rounding(out, dtype) + e * torch.finfo(dtype).eps


def check(got, want, bound, what):
    got = got.double().cpu()
    want, bound = want.cpu(), bound.cpu()
    off = (got - want).abs()
    bad = ~(off <= bound)  # a NaN fails
    if bad.any():
        i = int((off / bound.clamp(min=1e-300)).nan_to_num(nan=1e300).view(-1).argmax())
        at = [int(v) for v in torch.unravel_index(torch.tensor(i), got.shape)]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst at {at}: got "
                             f"{got.view(-1)[i]:.8g}, want {want.view(-1)[i]:.8g} +- {bound.view(-1)[i]:.3g}")
