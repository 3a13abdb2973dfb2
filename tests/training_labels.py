"""Cross entropy gradients at labels: inputs in which single products show D's entry at a label,
the entries in 64 bits, and bounds that count what the library rounds there.

Residual row b's label is Y[b % J].  Two blocks of J columns keep the entries apart from the
rest of the sums:
  columns j < J        the table is 0 there but for E[Y[j]][j], the residual rows are 0:
                       d_residual[b][b % J] = D[b][label] E[label][b % J], one product
  columns J <= j < 2J  the table is 0 there, residual row b only has a value at J + b % J:
                       d_table[Y[j]][J + j] = the sum of D[b][Y[j]] x[b][J + j] over the rows of label Y[j]
The other columns make the logits; a row is lifted towards its label until 1 - p is about 10^-u, u
from 0.5 to 6.  Rows b % 7 == 5 have no label, and nothing in the second block.
"""
import torch

EPS = {t: torch.finfo(t).eps for t in (torch.float32, torch.bfloat16, torch.float16)}


def make(n, V, d, dtype, seed=0):
    """(E, x, labels, Y) on the CPU."""
    gen = torch.Generator().manual_seed(7919 * seed + 31 * n + V + d)
    J = max(1, min(n, V, d // 4, 32))
    Y = torch.arange(J) * (V - 1) // max(J - 1, 1)
    b = torch.arange(n)
    E = torch.randn((V, d), generator=gen) * (0.3 / d ** 0.5)
    E[:, :2 * J] = 0
    E[Y] *= 4  # a label's row stands out, so that lifting a row towards it lifts few others
    E[Y, torch.arange(J)] = 1 + torch.rand(J, generator=gen)
    E = E.to(dtype)
    target = E[Y[b % J]].float()
    target[:, :2 * J] = 0
    u = 6.0 - 5.5 * (b % J % 8).float() / 7  # the same for a label's rows
    lift = torch.log(torch.tensor(float(max(V, 2)))) + u * 2.302585
    x = torch.randn((n, d), generator=gen)
    x += target * ((lift - (x * target).sum(1)) / target.square().sum(1))[:, None]
    x[:, :2 * J] = 0
    has = b % 7 != 5
    x[b[has], J + b[has] % J] = (1 + torch.rand(int(has.sum()), generator=gen)) * torch.where(b[has] % 3 == 0, -1.0, 1.0)
    labels = torch.where(has, Y[b % J], torch.full((n,), -100)).to(torch.int32)
    return E, x.to(dtype), labels, Y


def make_cancelling(n, V, d, dtype, seed=0):
    """(E, x, labels): the labels' logits are sums of large products that cancel, of columns d / 4 from
    either end, around the ordinary ones: an f32 accumulator loses 2^-9 and more of them.  The other
    table rows are 0 in those columns.  1 - p is about 10^-3 or less."""
    gen = torch.Generator().manual_seed(104729 * seed + 31 * n + V + d)
    q, y = d // 4, V // 2
    E = torch.randn((V, d), generator=gen) * (0.3 / d ** 0.5)
    E[y] *= 4
    E[:, :q], E[:, d - q:] = 0, 0
    E[y, :q] = 20 + 20 * torch.rand(q, generator=gen)
    E[y, d - q:] = E[y, :q]
    E = E.to(dtype)
    target = E[y].float().clone()
    target[:q], target[d - q:] = 0, 0
    x = torch.randn((n, d), generator=gen)
    lift = torch.log(torch.tensor(float(V))) + 7 + torch.rand(n, generator=gen) * 4
    x += target * ((lift - x @ target) / target.square().sum())[:, None]
    a = 20 + 20 * torch.rand((n, q), generator=gen)
    x[:, :q], x[:, d - q:] = a, -a
    return E, x.to(dtype), torch.full((n,), y, dtype=torch.int32)


def loss_of(E, x, labels):
    """(loss, lse, their bounds) in 64 bits where every row has a label.

    The label's logit is summed in 64 bits; the other logits are off by up to d * 2^-22 of their
    sums of magnitudes, which moves lse by their share 1 - p of it; exponentials, sums and joins as
    training_oracle.loss counts them (1e-5 for fewer than 100 additions in a row)."""
    xd, Ed = x.double(), E.double()
    L = xd @ Ed.t().contiguous()
    dL = x.shape[1] * 2.0 ** -22 * (xd.abs() @ Ed.abs().t().contiguous())
    at = labels.long()[:, None]
    dL.scatter_(1, at, 0.0)
    lse = torch.logsumexp(L, 1)
    loss = lse - L.gather(1, at)[:, 0]
    moved = -torch.expm1(-loss) * torch.expm1(dL.max(1).values) + 1e-5
    return loss, lse, moved + loss.abs() * 2.0 ** -24, moved + half_step(lse, torch.float32)


def entries(E, x, labels, lse, g, h=None):
    """(D at the labels, its bound) [n] in 64 bits for the given lse; 0 without a label.

    The label's logit is summed in 64 bits (d terms, 2^-52 of the sum of magnitudes is more than
    they lose); its distance to lse is rounded once to 32 bits, expm1 and exp are within 2 ulp, the
    products and the sum round once each: under 2^-21 of both terms.
    """
    has = labels >= 0
    rows = E[torch.where(has, labels, torch.zeros_like(labels)).long()].double()
    xd = x.double()
    t = (xd * rows).sum(1) - lse.double()
    g = g.double()
    h = torch.zeros_like(g) if h is None else h.double()
    first, second = g * torch.expm1(t), h * torch.exp(t)
    moved = x.shape[1] * 2.0 ** -52 * (xd * rows).abs().sum(1)
    e = 2.0 ** -21 * (first.abs() + second.abs()) + (g.abs() + h.abs()) * torch.exp(t) * moved
    zero = torch.zeros_like(t)
    return torch.where(has, first + second, zero), torch.where(has, e, zero)


def half_step(v, dtype):
    """Half the distance of the type's values at v (powers of two by frexp: a device's exp2 may round)."""
    smallest = {torch.float32: -126, torch.bfloat16: -126, torch.float16: -14}[dtype]
    v = v.abs().clamp(min=2.0 ** smallest)
    return v / torch.frexp(v).mantissa * (EPS[dtype] / 4)


def shown(E, x, labels, Y, entry, e_entry, rest_in_table):
    """(dx at [b][b % J], its bound, dE at [Y[j]][J + j], its bound); rows without a label: 0.

    f32: one product per row, rounded.  16 bits: D rounded to the type plus its rest in f32 (dx), the rest
    rounded to the type (dE up to 128 rows: eps^2 / 4 stays) or left out (eps / 2 stays).
    """
    n, J, dtype = x.shape[0], len(Y), x.dtype
    b = torch.arange(n)
    a = E[Y[b % J], b % J].double()
    has = labels >= 0
    dx = torch.where(has, entry * a, torch.zeros_like(a))
    e_dx = torch.where(has, e_entry * a + 2.0 ** -22 * dx.abs(), torch.zeros_like(a))
    xb = x[b, J + b % J].double()
    dE, e_dE = torch.zeros(J, dtype=torch.float64), torch.zeros(J, dtype=torch.float64)
    dE.index_add_(0, b % J, entry * xb)
    stays = 0.0 if dtype == torch.float32 else EPS[dtype] ** 2 / 4 if rest_in_table else EPS[dtype] / 2
    terms = (n + J - 1) // J + 2
    e_dE.index_add_(0, b % J, e_entry * xb.abs() + (stays + terms * 2.0 ** -22) * (entry * xb).abs())

    def rounded(v, e):
        return e + half_step(v.abs() + e, dtype)
    return dx, rounded(dx, e_dx), dE, rounded(dE, e_dE)


def pick(dx, dE, x, Y):
    """The same places of the library's outputs."""
    b = torch.arange(x.shape[0])
    J = len(Y)
    return dx[b, b % J], dE[Y, J + torch.arange(J)]


# every kernel that writes D: few rows and a small table (f32 D, by 16 x 16 and by larger tiles),
# 16 x 16 tiles with D in the table's type, 64, 128 and 256 columns, more than one piece
CASES = [("f32", 1, 300, 64), ("f32", 4, 4096, 256), ("bf16", 8, 3000, 136), ("f16", 3, 1000, 64),
         ("f32", 4, 70001, 64), ("bf16", 8, 40001, 64), ("f16", 5, 40001, 72),
         ("f32", 20, 4000, 128), ("bf16", 33, 3000, 136), ("f16", 64, 2000, 72),
         ("f32", 40, 40001, 100), ("bf16", 64, 20011, 264), ("f16", 37, 20011, 136),
         ("f32", 100, 9000, 256), ("bf16", 100, 40011, 264), ("f16", 128, 20001, 264),
         ("f32", 300, 20000, 600), ("bf16", 300, 30001, 520), ("f16", 700, 20001, 264),
         ("bf16", 40000, 9000, 32)]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def upstream(n, dtype, seed=0):
    """(g, h), no zeros: g about 1 / n, in f16 about 2^10, where entries of 1e-6 are not yet subnormal; h as a
    penalty on lse gives it."""
    gen = torch.Generator().manual_seed(seed + n)
    size = 1024.0 if dtype == torch.float16 else 1.0 / n
    return (0.5 + torch.rand(n, generator=gen)) * size, (torch.rand(n, generator=gen) - 0.5) * (1e-3 * size)


CANCELLING = [("f32", 4, 4096, 256), ("bf16", 8, 3000, 256), ("f32", 70, 20000, 512), ("f16", 64, 20011, 520),
              ("bf16", 100, 30001, 512), ("f16", 300, 9000, 1024), ("bf16", 300, 9000, 5376)]
