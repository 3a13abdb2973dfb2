"""Cross entropy over the vocabulary, its gradients and the gather's gradient on the GPU,
against their definitions in 64 bits (tests/training_oracle.py derives the tolerances)."""
import pytest
import torch

import embedding_table_gather_amd as etg
from tests import training_oracle as to
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODES = {torch.float32: etg.F32, torch.bfloat16: etg.BF16, torch.float16: etg.F16}


def make(n, V, d, dtype, seed=0, size=0.05):
    """(table, E, x, labels) on the GPU from CPU random numbers; labels in and outside the vocabulary."""
    g = torch.Generator().manual_seed(1000 * seed + 7 * n + V + d)
    E = (torch.randn((V, d), generator=g) * size).to(dtype).cuda()
    x = torch.randn((n, d), generator=g).to(dtype).cuda()
    labels = torch.randint(V, (n,), generator=g, dtype=torch.int64)
    if n > 2:
        labels[1] = -100
        labels[2] = V - 1
    if n > 5:
        labels[4], labels[5] = V, 2 ** 31 - 1
    return etg.Table(E, CODES[dtype], V, d), E, x, labels.to(torch.int32).cuda()


def upstream(n, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, generator=g) / max(n, 1)).cuda(), (torch.randn(n, generator=g) * 0.3 / max(n, 1)).cuda()


SHAPES = [(1, 1, 8), (1, 5, 8), (2, 300, 16), (3, 257, 72), (16, 256, 64), (64, 1000, 136), (65, 513, 200),
          (129, 700, 264), (257, 1031, 520), (300, 255, 1000), (513, 4097, 32)]
CASES = [(dtype, *shape) for dtype in sorted(TYPES) for shape in SHAPES] + \
    [("f32", 5, 100, 4), ("f32", 70, 515, 36)]  # 16-bit rows are multiples of 8 values


@pytest.mark.parametrize("dtype,n,V,d", CASES)
def test_loss(dtype, n, V, d):
    note(f"loss {dtype} {n} x {V} x {d}")
    t, E, x, labels = make(n, V, d, TYPES[dtype])
    loss, lse = t.cross_entropy(x, labels)
    torch.cuda.synchronize()
    assert loss.dtype == lse.dtype == torch.float32 and loss.shape == lse.shape == (n,)
    want, want_lse, tol, tol_lse = to.loss(x.cpu(), E.cpu(), labels.cpu())
    to.check(lse, want_lse, tol_lse, "lse")
    to.check(loss, want, tol, "loss")
    ok = to.has_label(labels, V)
    assert (loss[~ok] == 0).all()


@pytest.mark.parametrize("zloss", [False, True])
@pytest.mark.parametrize("dtype,n,V,d", CASES)
def test_grads(dtype, n, V, d, zloss):
    note(f"grads {dtype} {n} x {V} x {d}, zloss {zloss}")
    t, E, x, labels = make(n, V, d, TYPES[dtype])
    g, h = upstream(n)
    _, lse = t.cross_entropy(x, labels)
    dx, dE = t.cross_entropy_grad(x, labels, lse, g, h if zloss else None)
    torch.cuda.synchronize()
    assert dx.dtype == dE.dtype == x.dtype and dx.shape == x.shape and dE.shape == E.shape
    wx, wE, tx, tE = to.grads(x.cpu(), E.cpu(), labels.cpu(), lse.cpu(), g.cpu(), h.cpu() if zloss else None)
    to.check(dx, wx, tx, "residual gradient")
    to.check(dE, wE, tE, "table gradient")


def test_large_logits_and_far_tokens():
    # logits of hundreds, probabilities of 0 and 1, the largest token first and last
    n, V, d = 40, 777, 64
    for dtype in TYPES.values():
        note(f"large logits {dtype}")
        t, E, x, labels = make(n, V, d, dtype, seed=3, size=4.0)
        E[0], E[V - 1] = x[0] * 8, x[7] * 8
        loss, lse = t.cross_entropy(x, labels)
        dx, dE = t.cross_entropy_grad(x, labels, lse, 1 / n)
        torch.cuda.synchronize()
        want, want_lse, tol, tol_lse = to.loss(x.cpu(), E.cpu(), labels.cpu())
        to.check(lse, want_lse, tol_lse, "lse")
        to.check(loss, want, tol, "loss")
        wx, wE, tx, tE = to.grads(x.cpu(), E.cpu(), labels.cpu(), lse.cpu(), torch.full((n,), 1 / n))
        to.check(dx, wx, tx, "residual gradient")
        to.check(dE, wE, tE, "table gradient")


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_grads_against_differences(dtype):
    # (loss(x + e u) - loss(x - e u)) / 2e in 64 bits against <dx, u>; the same for the table.  The
    # difference's own error is e^2 / 6 times the third derivative, here below 1e-6 of the value
    n, V, d = 20, 300, 64
    t, E, x, labels = make(n, V, d, TYPES[dtype], seed=5, size=0.1)
    g, _ = upstream(n, 4)
    _, lse = t.cross_entropy(x, labels)
    dx, dE = t.cross_entropy_grad(x, labels, lse, g)
    torch.cuda.synchronize()
    E, x, labels, g = E.double().cpu(), x.double().cpu(), labels.cpu(), g.double().cpu()
    _, _, tx, tE = to.grads(x.to(TYPES[dtype]), E.to(TYPES[dtype]), labels, lse.cpu(), g)

    def total(x, E):
        L = x @ E.t()
        ok = to.has_label(labels, V)
        at = torch.where(ok, labels, torch.zeros_like(labels)).long()[:, None]
        return ((torch.logsumexp(L, 1) - L.gather(1, at)[:, 0]) * ok * g).sum()
    gen = torch.Generator().manual_seed(9)
    for _ in range(5):
        u, w = torch.randn(x.shape, generator=gen).double(), torch.randn(E.shape, generator=gen).double()
        e = 1e-4
        num = (total(x + e * u, E) - total(x - e * u, E)) / (2 * e)
        got = (dx.double().cpu() * u).sum()
        assert abs(num - got) <= (tx * u.abs()).sum() + 1e-6 * (dx.double().cpu() * u).abs().sum()
        num = (total(x, E + e * w) - total(x, E - e * w)) / (2 * e)
        got = (dE.double().cpu() * w).sum()
        assert abs(num - got) <= (tE * w.abs()).sum() + 1e-6 * (dE.double().cpu() * w).abs().sum()


def test_grad_loss_number_and_single_outputs():
    n, V, d = 50, 600, 128
    t, E, x, labels = make(n, V, d, torch.bfloat16, seed=2)
    _, lse = t.cross_entropy(x, labels)
    dx, dE = t.cross_entropy_grad(x, labels, lse, torch.full((n,), 0.25, device="cuda"))
    a, b = t.cross_entropy_grad(x, labels, lse, 0.25)
    only_x, none = t.cross_entropy_grad(x, labels, lse, 0.25, table_grad=False)
    none2, only_E = t.cross_entropy_grad(x, labels, lse, 0.25, residual_grad=False)
    torch.cuda.synchronize()
    assert none is None and none2 is None
    for p, q in ((dx, a), (dE, b), (dx, only_x), (dE, only_E)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_accumulate(dtype):
    n, V, d = 70, 513, 72
    t, E, x, labels = make(n, V, d, TYPES[dtype], seed=8)
    g, h = upstream(n, 1)
    _, lse = t.cross_entropy(x, labels)
    old = (torch.randn((V, d), generator=torch.Generator().manual_seed(1)) * 0.1).to(TYPES[dtype]).cuda()
    out = old.clone()
    _, got = t.cross_entropy_grad(x, labels, lse, g, h, out_table=out, accumulate=True)
    torch.cuda.synchronize()
    assert got is out
    _, wE, _, tE = to.grads(x.cpu(), E.cpu(), labels.cpu(), lse.cpu(), g.cpu(), h.cpu(), old.cpu())
    to.check(out, wE, tE, "table gradient")


def test_rows_without_a_target():
    n, V, d = 9, 300, 64
    for dtype in TYPES.values():
        note(f"no targets {dtype}")
        t, E, x, _ = make(n, V, d, dtype, seed=6)
        labels = torch.tensor([-1, -100, V, V + 1, 2 ** 31 - 1, -2 ** 31, -1, -1, -1], dtype=torch.int32).cuda()
        loss, lse = t.cross_entropy(x, labels)
        dx, dE = t.cross_entropy_grad(x, labels, lse, 1.0)
        h = upstream(n)[1]
        zx, zE = t.cross_entropy_grad(x, labels, lse, 1.0, h)  # what reaches lse still flows
        torch.cuda.synchronize()
        assert not loss.any() and not dx.any() and not dE.any() and torch.isfinite(lse).all()
        wx, wE, tx, tE = to.grads(x.cpu(), E.cpu(), labels.cpu(), lse.cpu(), torch.zeros(n), h.cpu())
        to.check(zx, wx, tx, "residual gradient")
        to.check(zE, wE, tE, "table gradient")


def test_nan_and_infinite_logits():
    n, V, d = 6, 600, 64
    t, E, x, labels = make(n, V, d, torch.bfloat16, seed=4)
    x[0, 3] = float("nan")            # a whole row of NaN logits
    loss, lse = t.cross_entropy(x, torch.tensor([1, 2, -1, 3, 4, 5], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert torch.isnan(lse[0]) and torch.isnan(loss[0]) and torch.isfinite(lse[1:]).all() and loss[2] == 0
    # a table row of the type's lowest value: logits of -inf (overflow) weigh nothing
    t, E, x, labels = make(n, V, d, torch.float32, seed=4)
    x = x.abs() + 4.0
    E[300] = torch.finfo(torch.float32).min
    labels = torch.arange(n, dtype=torch.int32, device="cuda")
    loss, lse = t.cross_entropy(x, labels)
    rest = torch.cat([E[:300], E[301:]])
    want, want_lse, tol, tol_lse = to.loss(x.cpu(), rest.cpu(), labels.cpu())
    torch.cuda.synchronize()
    to.check(lse, want_lse, tol_lse, "lse")
    to.check(loss, want, tol, "loss")
    # a single NaN logit among finite ones, in each tile of the vocabulary
    for v in (0, 255, 256, 599):
        t, E, x, labels = make(n, V, d, torch.float16, seed=4)
        E[v, 0] = float("nan")
        loss, lse = t.cross_entropy(x, labels)
        torch.cuda.synchronize()
        assert torch.isnan(lse).all()


@pytest.mark.parametrize("dtype,pad,offset", [("bf16", 0, 1), ("bf16", 3, 0), ("f16", 8, 8), ("f16", 1, 5),
                                               ("f32", 1, 1), ("f32", 4, 0)])
def test_strided_and_unaligned_rows(dtype, pad, offset):
    n, V, d = 37, 520, 136
    t, E, x, labels = make(n, V, d, TYPES[dtype], seed=11)
    buf = torch.full((n * (d + pad) + offset,), float("nan"), dtype=x.dtype, device="cuda")
    xs = buf[offset:].view(n, d + pad)[:, :d]
    xs.copy_(x)
    outbuf = torch.full((n * (d + pad) + offset,), 7.0, dtype=x.dtype, device="cuda")
    out = outbuf[offset:].view(n, d + pad)[:, :d]
    g, h = upstream(n, 3)
    note(f"strided {dtype} {pad} {offset}")
    loss, lse = t.cross_entropy(x, labels)
    dx, dE = t.cross_entropy_grad(x, labels, lse, g, h)
    loss2, lse2 = t.cross_entropy(xs, labels)
    dx2, dE2 = t.cross_entropy_grad(xs, labels, lse, g, h, out_residual=out)
    torch.cuda.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2) and torch.equal(dx, dx2) and torch.equal(dE, dE2)
    assert (outbuf[offset:].view(n, d + pad)[:, d:] == 7).all() and (outbuf[:offset] == 7).all()


def test_far_rows():
    # rows more than 8 MiB apart are packed first
    n, V, d = 3, 40, 64
    t, E, x, labels = make(n, V, d, torch.bfloat16, seed=12)
    far = torch.zeros((n, 9 << 20), dtype=torch.bfloat16, device="cuda")
    far[:, :d] = x
    a = t.cross_entropy(x, labels)
    b = t.cross_entropy(far[:, :d], labels)
    ga = t.cross_entropy_grad(x, labels, a[1], 0.5)
    gb = t.cross_entropy_grad(far[:, :d], labels, a[1], 0.5)
    torch.cuda.synchronize()
    for p, q in zip(a + ga, b + gb):
        assert torch.equal(p, q)


def test_pieces_of_the_vocabulary():
    # 65,536 residual rows: the backward pass takes 2,048 table rows at a time, the forward one
    # 131,072; checked on some rows and all of the table's gradient in 64 bits on the GPU
    n, V, d = 65536, 5000, 16
    t, E, x, labels = make(n, V, d, torch.bfloat16, seed=13)
    g, h = upstream(n, 5)
    note("pieces, backward")
    loss, lse = t.cross_entropy(x, labels)
    dx, dE = t.cross_entropy_grad(x, labels, lse, g, h)
    torch.cuda.synchronize()
    want, want_lse, tol, tol_lse = to.loss(x, E, labels)
    to.check(loss, want, tol, "loss")
    wx, wE, tx, tE = to.grads(x, E, labels, lse, g, h)
    to.check(dx, wx, tx, "residual gradient")
    to.check(dE, wE, tE, "table gradient")
    del want, want_lse, tol, tol_lse, wx, wE, tx, tE
    note("pieces, forward")
    V = 140001
    t, E, x, labels = make(n, V, 8, torch.float16, seed=14)
    loss, lse = t.cross_entropy(x, labels)
    torch.cuda.synchronize()
    some = torch.arange(0, n, 37, device="cuda")
    want, want_lse, tol, tol_lse = to.loss(x[some], E, labels[some])
    # 547 tiles in turn over 64 lanes and two pieces: still fewer than 100 additions in a row
    to.check(lse[some], want_lse, tol_lse, "lse")
    to.check(loss[some], want, tol, "loss")


def test_empty_batch():
    V, d = 300, 64
    t, E, _, _ = make(4, V, d, torch.bfloat16)
    x, labels = E[:0], torch.empty(0, dtype=torch.int32, device="cuda")
    loss, lse = t.cross_entropy(x, labels)
    assert loss.shape == lse.shape == (0,)
    out = torch.full((V, d), 3.0, dtype=torch.bfloat16, device="cuda")
    dx, dE = t.cross_entropy_grad(x, labels, lse, 1.0, out_table=out)
    torch.cuda.synchronize()
    assert dx.shape == (0, d) and dE is out and not out.any()
    out.fill_(3.0)
    t.cross_entropy_grad(x, labels, lse, 1.0, out_table=out, accumulate=True)
    torch.cuda.synchronize()
    assert (out == 3).all()


ROWS = [(1, 1, 8), (1, 100, 16), (7, 3, 64), (64, 64, 256), (65, 40, 264), (628, 1000, 896), (1000, 1, 72),
        (4096, 300, 64), (4097, 300, 64), (8192, 5000, 16), (8193, 5000, 16), (20000, 300001, 8), (30011, 50, 520)]


@pytest.mark.parametrize("kind", ["uniform", "heavy", "same"])
@pytest.mark.parametrize("gtype,dtype", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"),
                                         ("bf16", "f32")])
@pytest.mark.parametrize("n,V,d", ROWS)
def test_gather_grad(n, V, d, gtype, dtype, kind):
    note(f"gather grad {n} x {V} x {d} {gtype} -> {dtype}, {kind}")
    g = torch.Generator().manual_seed(n + V + d)
    ids = torch.randint(V, (n,), generator=g)
    if kind == "heavy":
        ids[torch.rand(n, generator=g) < 0.5] = V // 2
    if kind == "same":
        ids[:] = V - 1
    if n > 3 and kind != "same":
        ids[0], ids[n // 2], ids[n - 1] = -1, V, 2 ** 31 - 1
    ids = ids.to(torch.int32).cuda()
    grad = torch.randn((n, d), generator=g).to(TYPES[gtype]).cuda()
    t = etg.Table(torch.zeros((V, d), dtype=TYPES[dtype], device="cuda"), CODES[TYPES[dtype]], V, d)
    out = torch.full((V, d), float("nan"), dtype=TYPES[dtype], device="cuda")
    got = t.embed_gather_grad(grad, ids, scale="sqrt_d", out=out)
    old = torch.randn((V, d), generator=g).to(TYPES[dtype]).cuda()
    added = t.embed_gather_grad(grad, ids, scale=-0.5, out=old.clone(), accumulate=True)
    torch.cuda.synchronize()
    assert got is out
    want, tol = to.gather_grad(grad, ids, V, etg.sqrt_d(d), TYPES[dtype])
    to.check(got, want, tol, "gradient")
    want, tol = to.gather_grad(grad, ids, V, -0.5, TYPES[dtype], old)
    to.check(added, want, tol, "added gradient")
    untouched = torch.ones(V, dtype=torch.bool)
    i = ids.cpu().long()
    untouched[i[(i >= 0) & (i < V)]] = False
    assert torch.equal(added.cpu()[untouched], old.cpu()[untouched]) and not got.cpu()[untouched].any()


def test_gather_grad_f32_out_odd_width_and_strides():
    # a f32 output beside a 16-bit table; rows of 4 values more than a multiple of 8; strided gradients
    V, n = 90, 333
    g = torch.Generator().manual_seed(2)
    ids = torch.randint(-3, V + 3, (n,), generator=g, dtype=torch.int32).cuda()
    for dtype, d, gtype, pad in ((torch.bfloat16, 72, torch.float32, 1), (torch.float16, 8, torch.float16, 3),
                                 (torch.float32, 36, torch.bfloat16, 1), (torch.float32, 4, torch.float16, 0)):
        note(f"gather grad f32 out, {dtype} {d} {gtype}")
        t = etg.Table(torch.zeros((V, d), dtype=dtype, device="cuda"), CODES[dtype], V, d)
        buf = torch.full((n, d + pad), float("nan"), dtype=gtype, device="cuda")
        buf[:, :d] = torch.randn((n, d), generator=g).cuda()
        grad = buf[:, :d]
        got = t.embed_gather_grad(grad, ids, out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert got.dtype == torch.float32
        want, tol = to.gather_grad(grad, ids, V, 1.0, torch.float32)
        to.check(got, want, tol, "gradient")


def test_gather_grad_of_nothing():
    V, d = 50, 64
    t = etg.Table(torch.zeros((V, d), dtype=torch.bfloat16, device="cuda"), etg.BF16, V, d)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    out = torch.full((V, d), 2.0, dtype=torch.bfloat16, device="cuda")
    t.embed_gather_grad(torch.empty((0, d), device="cuda"), none, out=out, accumulate=True)
    torch.cuda.synchronize()
    assert (out == 2).all()
    t.embed_gather_grad(torch.empty((0, d), device="cuda"), none, out=out)
    torch.cuda.synchronize()
    assert not out.any()
    bad = torch.full((100,), -1, dtype=torch.int32, device="cuda")
    out.fill_(2.0)
    t.embed_gather_grad(torch.full((100, d), float("nan"), device="cuda"), bad, out=out, accumulate=True)
    torch.cuda.synchronize()
    assert (out == 2).all()


def test_gather_grad_is_the_gathers():
    # <gather(E), G> is linear in E: its difference quotient along W is <gather_grad(G), W>
    V, d, n = 700, 64, 5000
    g = torch.Generator().manual_seed(21)
    W = torch.randn((V, d), generator=g).cuda()
    ids = torch.randint(V, (n,), generator=g, dtype=torch.int32).cuda()
    G = torch.randn((n, d), generator=g).cuda()
    t = etg.Table(W, etg.F32, V, d)
    rows = t.embed_gather(ids, scale="sqrt_d")
    dW = t.embed_gather_grad(G, ids, scale="sqrt_d")
    a, b = (rows.double() * G.double()).sum(), (dW.double() * W.double()).sum()
    _, tol = to.gather_grad(G, ids, V, etg.sqrt_d(d), torch.float32)
    # the gathered rows are rounded once
    assert abs(a - b) <= (tol * W.double().abs()).sum() + 2.0 ** -24 * (rows.double() * G.double()).abs().sum()


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_training_steps_of_a_tied_table(dtype):
    """Gather, a body of one product, loss, gradients, the gather's gradient added to the tied
    table's, as a user runs them: three steps, each against 64 bits from the same weights."""
    V, d, n = 1500, 128, 96
    T = TYPES[dtype]
    g = torch.Generator().manual_seed(31)
    E = (torch.randn((V, d), generator=g) * 0.05).to(T).cuda()
    W = (torch.randn((d, d), generator=g) / d ** 0.5).cuda()
    tokens = torch.randint(V, (n + 1,), generator=g, dtype=torch.int32).cuda()
    t = etg.Table(E, CODES[T], V, d)
    for step in range(3):
        ids, labels = tokens[:-1].contiguous(), tokens[1:].contiguous()
        note(f"tied step {step} {dtype}")
        x0 = t.embed_gather(ids, scale="sqrt_d")
        x = (x0 @ W).to(T)
        loss, lse = t.cross_entropy(x, labels)
        dx, dE = t.cross_entropy_grad(x, labels, lse, 1 / n)
        before = dE.clone()
        dx0 = dx.float() @ W.t()
        t.embed_gather_grad(dx0, ids, scale="sqrt_d", out=dE, accumulate=True)
        torch.cuda.synchronize()
        want, _, tol, _ = to.loss(x, E, labels)
        to.check(loss, want, tol, "loss")
        wx, wE, tx, tE = to.grads(x, E, labels, lse, torch.full((n,), 1 / n, device="cuda"))
        to.check(dx, wx, tx, "residual gradient")
        to.check(before, wE, tE, "table gradient of the head")
        wE, tE = to.gather_grad(dx0, ids, V, etg.sqrt_d(d), T, before)
        to.check(dE, wE, tE, "table gradient")
        E -= (0.5 * dE.float()).to(T)
        W -= 0.1 * (x0.t().contiguous() @ dx.float())
        tokens = tokens.roll(1)


def test_repeats_bitwise_and_on_other_streams():
    n, V, d = 200, 3001, 264
    t, E, x, labels = make(n, V, d, torch.bfloat16, seed=41)
    ids = torch.randint(-2, 50, (n * 3,), dtype=torch.int32, device="cuda")
    grad = torch.randn((n * 3, d), device="cuda")
    g, h = upstream(n, 6)

    def all_of_it():
        loss, lse = t.cross_entropy(x, labels)
        dx, dE = t.cross_entropy_grad(x, labels, lse, g, h)
        return loss, lse, dx, dE, t.embed_gather_grad(grad, ids, scale=2.0)
    first = all_of_it()
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for rep in range(3):  # three streams at once, each with workspaces of its own
        for s in side:
            with torch.cuda.stream(s):
                got.append(all_of_it())
    torch.cuda.synchronize()
    for outs in got:
        for a, b in zip(first, outs):
            assert torch.equal(a, b)


def test_captured_graph_replays():
    n, V, d = 100, 2000, 136
    t, E, x, labels = make(n, V, d, torch.float16, seed=43)
    ids = torch.randint(-2, V, (9000,), dtype=torch.int32, device="cuda")
    grad = torch.randn((9000, d), device="cuda")
    dE = torch.zeros((V, d), dtype=torch.float16, device="cuda")
    outs = {}

    def step():
        loss, lse = t.cross_entropy(x, labels)
        dx, _ = t.cross_entropy_grad(x, labels, lse, 0.01, out_table=dE)
        t.embed_gather_grad(grad, ids, scale=0.01, out=dE, accumulate=True)
        return loss, lse, dx
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs["a"] = step()
    with torch.cuda.graph(other, stream=side):
        outs["b"] = step()
    for rep in range(4):
        x.copy_(torch.randn((n, d), generator=torch.Generator().manual_seed(rep)).to(x.dtype))
        ids.copy_(ids.roll(17))
        want = [v.clone() for v in step()] + [dE.clone()]
        torch.cuda.synchronize()
        for name, gr in (("a", graph), ("b", other)):
            dE.fill_(float("nan"))
            gr.replay()
            torch.cuda.synchronize()
            for a, b in zip(want, list(outs[name]) + [dE]):
                assert torch.equal(a, b), (rep, name)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("n,V", [(3, 300), (8, 5000), (40, 700), (100, 2000), (150, 513), (600, 1100)])
def test_padding_may_hold_anything(dtype, n, V):
    # rows without a target, or whose gradient is 0, hold NaN and infinities: as if they were 0
    note(f"padding {dtype} {n} x {V}")
    d = 72
    t, E, x, labels = make(n, V, d, TYPES[dtype], seed=51)
    g = upstream(n, 3)[0]
    dead = torch.arange(n, device="cuda") % 3 == 1
    labels[dead] = -100
    labels[0], g[0], dead[0] = 1, 0.0, True
    clean = torch.where(dead[:, None], torch.zeros_like(x), x)
    bad = x.clone()
    bad[dead] = torch.tensor([float("nan"), float("inf"), float("-inf")], device="cuda").repeat(24).to(x.dtype)
    want_loss, want_lse = t.cross_entropy(clean, labels)
    loss, lse = t.cross_entropy(bad, labels)
    want = t.cross_entropy_grad(clean, labels, want_lse, g)
    got = t.cross_entropy_grad(bad, labels, lse, g)
    only_x, _ = t.cross_entropy_grad(bad, labels, lse, g, table_grad=False)
    torch.cuda.synchronize()
    live = ~dead
    assert torch.equal(loss[live], want_loss[live]) and torch.equal(lse[live], want_lse[live])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(only_x, want[0])
    assert not got[0][dead].any()


# more tiles than CUs in each product, odd numbers of stages; many labels in one tile
@pytest.mark.parametrize("dtype,n,V,d", [("bf16", 700, 40001, 520), ("f16", 700, 40001, 520), ("f32", 600, 24003, 524),
                                         ("bf16", 128, 40001, 264), ("f16", 65, 30000, 264), ("bf16", 100, 20011, 328),
                                         ("bf16", 8, 150001, 64), ("f16", 8, 300003, 64), ("f32", 8, 20001, 1000)])
def test_more_tiles_than_units(dtype, n, V, d):
    note(f"many tiles {dtype} {n} x {V} x {d}")
    t, E, x, labels = make(n, V, d, TYPES[dtype], seed=52)
    labels[n // 2:] = torch.where(labels[n // 2:] % 2 == 0, 17, labels[n // 2:])  # one token many times
    g, h = upstream(n, 8)
    loss, lse = t.cross_entropy(x, labels)
    old = (torch.randn((V, d), generator=torch.Generator().manual_seed(2)) * 0.01).to(x.dtype).cuda()
    out = old.clone()
    dx, dE = t.cross_entropy_grad(x, labels, lse, g, h)
    t.cross_entropy_grad(x, labels, lse, g, h, out_table=out, accumulate=True)
    torch.cuda.synchronize()
    want, want_lse, tol, tol_lse = to.loss(x, E, labels)
    # tiles in turn over 64 lanes: fewer than 100 additions in a row
    to.check(lse, want_lse, tol_lse, "lse")
    to.check(loss, want, tol, "loss")
    wx, wE, tx, tE = to.grads(x, E, labels, lse, g, h)
    to.check(dx, wx, tx, "residual gradient")
    to.check(dE, wE, tE, "table gradient")
    _, wE, _, tE = to.grads(x, E, labels, lse, g, h, old)
    to.check(out, wE, tE, "table gradient, added")


@pytest.mark.parametrize("n", [3, 70, 260])
def test_table_past_4_gib(n):
    # 4.5 GB of bf16 rows; labels and ids at both ends
    V, d = 420001, 5376
    note(f"4.5 GB table, {n} rows")
    gen = torch.Generator(device="cuda").manual_seed(61)
    E = (torch.randn((V, d), generator=gen, device="cuda", dtype=torch.bfloat16) * 0.02)
    x = torch.randn((n, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    labels = torch.randint(V, (n,), generator=gen, device="cuda").to(torch.int32)
    labels[0], labels[1], labels[2] = V - 1, 0, V - 300
    g, h = upstream(n, 9)
    t = etg.Table(E, etg.BF16, V, d)
    loss, lse = t.cross_entropy(x, labels)
    dx, dE = t.cross_entropy_grad(x, labels, lse, g, h)
    torch.cuda.synchronize()
    want, want_lse, tol, tol_lse = to.loss(x, E, labels)
    # 1,641 tiles in turn over 64 lanes: 26 additions and six exchanges
    to.check(lse, want_lse, tol_lse, "lse")
    to.check(loss, want, tol, "loss")
    del want, want_lse, tol, tol_lse
    note("  gradients")
    wx, _, tx, _ = to.grads(x, E, labels, lse, g, h) if n == 3 else (None,) * 4
    if wx is not None:
        to.check(dx, wx, tx, "residual gradient")
    del wx, tx
    # the table's gradient at rows near the start, the 4 GiB border and the end, and at the labels
    some = torch.cat([torch.arange(70), torch.arange(399400, 399500), torch.arange(V - 320, V),
                      labels.long().cpu()]).unique().cuda()
    ok = torch.isin(some, labels.long())
    assert ok.sum() >= 3
    L = x.double() @ E[some].double().t().contiguous()
    hot = (labels.long()[:, None] == some[None, :]).double()
    # as the oracle's gradients: the product with D, its rounding to 8 bits and the logits' error
    cp = torch.exp(L - lse.double()[:, None]) * (g + h).double()[:, None]
    D = cp - hot * g.double()[:, None]
    dL = d * 2.0 ** -22 * (x.double().abs() @ E[some].double().abs().t().contiguous())
    dD = cp.abs() * (torch.expm1(dL) + 4e-6) + 2.0 ** -23 * (cp.abs() + hot * g.double().abs()[:, None])
    dD = dD + D.abs() * 2.0 ** -8 + to.SUBNORMAL[torch.bfloat16] / 2
    want = D.t().contiguous() @ x.double()
    e = dD.t().contiguous() @ x.double().abs() + (n + 1) * 2.0 ** -22 * ((D.abs() + dD).t().contiguous() @ x.double().abs())
    to.check(dE[some], want, e + to.rounding(want, torch.bfloat16) + e * 2.0 ** -7, "table gradient")
    note("  gather's gradient")
    ids = torch.cat([labels, labels, torch.tensor([-1, V], dtype=torch.int32, device="cuda")])
    grad = torch.randn((len(ids), d), generator=gen, device="cuda", dtype=torch.bfloat16)
    t.embed_gather_grad(grad, ids, scale=3.0, out=dE)
    torch.cuda.synchronize()
    want, tol = to.gather_grad(grad[:, :], torch.searchsorted(some, ids.long()).where((ids >= 0) & (ids < V), -1).to(torch.int32),
                               len(some), 3.0, torch.bfloat16)
    to.check(dE[some], want, tol, "gather's gradient")
    assert int((dE != 0).any(1).sum()) == int(labels.unique().numel())


@pytest.mark.parametrize("n,V,d", [(70001, 3000, 32), (140000, 200000, 16), (70000, 20, 1032)])
def test_gather_grad_of_many_ids(n, V, d):
    note(f"{n} ids into {V} x {d}")
    gen = torch.Generator(device="cuda").manual_seed(71)
    t = etg.Table(torch.zeros((V, d), dtype=torch.bfloat16, device="cuda"), etg.BF16, V, d)
    ids = torch.randint(-2, V + 2, (n,), generator=gen, device="cuda").to(torch.int32)
    grad = torch.randn((n, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    old = torch.randn((V, d), generator=gen, device="cuda")
    got, added = t.embed_gather_grad(grad, ids, out_dtype=etg.F32), old.clone()
    t.embed_gather_grad(grad, ids, out=added, accumulate=True)
    torch.cuda.synchronize()
    to.check(got, *to.gather_grad(grad, ids, V, 1.0, torch.float32), "rows")
    to.check(added, *to.gather_grad(grad, ids, V, 1.0, torch.float32, old), "rows, added")


def test_two_graphs_share_a_workspace():
    # replayed one after the other on a stream: each leaves what it leaves when run alone
    n, V, d = 150, 3000, 136
    t, E, x, labels = make(n, V, d, torch.bfloat16, seed=81)
    g = upstream(n, 2)[0]
    _, lse = t.cross_entropy(x, labels)
    _, lse2 = t.cross_entropy(x[:20], labels[:20])
    L = etg.lib()
    need = max(L.etg_cross_entropy_grad_workspace(t._h, n), L.etg_cross_entropy_grad_workspace(t._h, 20))
    space = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = [v.clone() for v in t.cross_entropy_grad(x, labels, lse, g) + t.cross_entropy_grad(x[:20], labels[:20], lse2, 0.5)]
    side = torch.cuda.Stream()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    torch.cuda.synchronize()
    with torch.cuda.graph(graphs[0], stream=side):
        outs += t.cross_entropy_grad(x, labels, lse, g, workspace=space)
    with torch.cuda.graph(graphs[1], stream=side):
        outs += t.cross_entropy_grad(x[:20], labels[:20], lse2, 0.5, workspace=space)
    for rep in range(3):
        space.fill_(255)
        for v in outs:
            v.fill_(7)
        graphs[rep % 2].replay()
        graphs[1 - rep % 2].replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b), rep


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,V,d", [(20, 300, 64), (70, 2000, 136), (128, 700, 72), (200, 3001, 264), (700, 300, 128),
                                   (5000, 600, 64)])
def test_label_entries_keep_what_rounding_takes(dtype, n, V, d):
    # D is rounded to 16 bits, but what that takes from a label's entry is added again, to the table's
    # gradient up to 128 rows: the bound without that part of it (of a rest that is itself
    # rounded: eps^2 / 4 of the entry).  Few distinct labels, many of them in one tile
    note(f"rests {dtype} {n} x {V} x {d}")
    t, E, x, labels = make(n, V, d, TYPES[dtype], seed=91, size=0.02)
    labels[n // 2:] = (labels[n // 2:] & 3) * 64 + 5
    g = upstream(n, 11)[0]
    _, lse = t.cross_entropy(x, labels)
    dx, dE = t.cross_entropy_grad(x, labels, lse, g)
    torch.cuda.synchronize()
    wx, wE, tx, tE = to.grads(x, E, labels, lse, g)
    ok = to.has_label(labels, V)
    at = labels[ok].long()
    p = torch.exp((x.double() @ E.double().t().contiguous())[ok, at] - lse.double()[ok])
    entry = (g.double()[ok] * (p - 1)).abs() * (torch.finfo(x.dtype).eps / 2 - torch.finfo(x.dtype).eps ** 2 / 4)
    less_x, less_E = torch.zeros_like(tx), torch.zeros_like(tE)
    less_x[ok] = entry[:, None] * E.double().abs()[at]
    less_E.index_add_(0, at, entry[:, None] * x.double().abs()[ok])
    to.check(dx, wx, tx - less_x, "residual gradient")
    to.check(dE, wE, tE - less_E if n <= 128 else tE, "table gradient")
