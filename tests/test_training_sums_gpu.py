"""Cross entropy gradients under inputs that show every row's share of the sums
(tests/training_sums.py), on small tables and on one past 4 GiB."""
import pytest
import torch

import embedding_table_gather_amd as etg
from tests import training_sums as ts
from tests.gpu_util import note

pytestmark = pytest.mark.gpu
CODES = {torch.float32: etg.F32, torch.bfloat16: etg.BF16, torch.float16: etg.F16}


def _check(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}"


def _run(n, V, d, dtype, device):
    E, x, labels, h = ts.make(n, V, d, dtype, device)
    E, x, labels, h = E.cuda(), x.cuda(), labels.cuda(), h.cuda()
    half = d // 2
    t = etg.Table(E, CODES[dtype], V, d)
    loss, lse = t.cross_entropy(x, labels)
    dx, dE = t.cross_entropy_grad(x, labels, lse, 1.0, h)
    torch.cuda.synchronize()
    assert not loss.any()
    wx, wE = ts.want(E, x, h)
    _check(dx[:, 1:half], wx, ts.bound(wx, n, V, d, dtype), "residual gradient")
    assert not dx[:, half:].any()
    row = wE[None, :].expand(V, -1)
    tE = ts.bound(wE, n, V, d, dtype)
    for v in range(0, V, 20000):
        _check(dE[v:v + 20000, half:], row[v:v + 20000], tE, "table gradient")
        assert not dE[v:v + 20000, 1:half].any()
    if ts.exact_d(n, V, d, dtype):  # added to what is there: twice, exactly
        again = dE.clone()
        t.cross_entropy_grad(x, labels, lse, 1.0, h, residual_grad=False, out_table=again, accumulate=True)
        torch.cuda.synchronize()
        want = (dE[0].double() + torch.cat([torch.zeros(half, dtype=torch.float64, device="cuda"), wE])).to(dtype)
        want[0] = again[0, 0]
        assert all(torch.equal(again[v:v + 20000, 1:], want[None, 1:].expand(len(again[v:v + 20000]), -1))
                   for v in range(0, V, 20000))


@pytest.mark.parametrize("case", ts.CASES, ids=str)
def test_every_row_counts(case):
    note(f"sums {case}")
    dtype, n, V, d = ts.TYPES[case[0]], *case[1:]
    _run(n, V, d, dtype, "cpu")


@pytest.mark.parametrize("n", [3, 70, 260])
def test_every_row_of_a_table_past_4_gib_counts(n):
    note(f"sums, 4.5 GB table, {n} rows")
    _run(n, 420001, 5376, torch.bfloat16, "cuda")


@pytest.mark.parametrize("dtype", sorted(ts.TYPES))
@pytest.mark.parametrize("n,V,d", [(1, 7, 64), (4, 4096, 256), (60, 20011, 64), (100, 3001, 72), (300, 70001, 136)])
def test_lse_near_zero(dtype, n, V, d):
    """Logits that are exact in f32 (one product each), with lse within about 1 of 0: what is left are the
    exponentials, within 2^-23 (1 + |distance to the largest|) each, the additions, at most 64 + V / 16384 in
    a row, the logarithm and one rounding."""
    note(f"lse near zero {dtype} {n} x {V} x {d}")
    T = ts.TYPES[dtype]
    gen = torch.Generator().manual_seed(n + V + d)
    E = torch.randn((V, d), generator=gen)
    shift = round(float(torch.log(torch.tensor(float(V)))) * 16) / 16 + 0.75
    E[:, 0] = torch.randint(-32, 33, (V,), generator=gen) / 16 - shift
    E = E.to(T)
    x = torch.zeros((n, d))
    x[:, 0] = 1 - (torch.arange(n) % 2) / 4
    x = x.to(T)
    labels = torch.randint(V, (n,), generator=gen, dtype=torch.int32)
    t = etg.Table(E.cuda(), CODES[T], V, d)
    loss, lse = t.cross_entropy(x.cuda(), labels.cuda())
    torch.cuda.synchronize()
    L = x[:, :1].double() * E[:, 0].double()[None, :]
    want = torch.logsumexp(L, 1)
    assert want.abs().max() < 4.5
    far = float((L.max(1, keepdim=True).values - L).max())
    e = (1 + far) * 2.0 ** -23 + (64 + V / 16384) * 2.0 ** -24
    _check(lse.cpu(), want, e + ts.half_step(want.abs() + e, torch.float32), "lse")
    want = want - L.gather(1, labels.long()[:, None])[:, 0]
    _check(loss.cpu(), want, e + ts.half_step(want.abs() + e, torch.float32), "loss")


@pytest.mark.parametrize("n,V,d", [(21, 5000, 64), (42, 20011, 136), (150, 5000, 264), (300, 9001, 72)])
def test_f16_rows_of_small_gradients(n, V, d):
    """Row b's gradient is 2^-(b % 21) of the largest: D is kept in f16 times one power of two, which puts the
    largest coefficient at 2^13 or more, so an entry is off by 2^-11 of itself or half of f16's smallest step,
    2^-25 / 2^13 of that coefficient, and by 1e-5 of itself before; sums of V terms round by 2^-22 each at most."""
    note(f"small gradients {n} x {V} x {d}")
    T = torch.float16
    E, x, labels, _ = ts.make(n, V, d, T)
    half = d // 2
    k = torch.arange(n) % 21
    h = (1000.0 * (1 + torch.arange(n) / (3.0 * n)) * 0.5 ** k.double()).float()
    t = etg.Table(E.cuda(), etg.F16, V, d)
    _, lse = t.cross_entropy(x.cuda(), labels.cuda())
    dx, _ = t.cross_entropy_grad(x.cuda(), labels.cuda(), lse, 0.0, h.cuda(), table_grad=False)
    both, _ = t.cross_entropy_grad(x.cuda(), labels.cuda(), lse, 0.0, h.cuda())
    torch.cuda.synchronize()
    assert torch.equal(dx, both)
    D, sums = h.double() / V, E[:, 1:half].double().sum(0)
    e = D * (1e-5 + 2.0 ** -11 + (V + 64) * 2.0 ** -22) + 2.0 ** -38 * float(h.max())
    want, bound = D[:, None] * sums[None, :], e[:, None] * sums[None, :]
    _check(dx[:, 1:half].cpu(), want, bound + ts.half_step(want + bound, T), "residual gradient")
