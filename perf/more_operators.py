"""Cases of the training operators of a tied table: Table.cross_entropy, Table.cross_entropy_grad,
Table.embed_gather_grad.

Each case is one call of a training or evaluation loop, or the three calls of a step.  ``run``
computes it either through this package (``own`` true) or in a plain form of elementary torch
operations (``own`` false).
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    """The shapes are this package's own configurations (262,144 x 5,376, x 5,120 and x 768, 151,936 x
    896, 4,096 x 256) and generic odd ones."""
    return [
        # the tiny configuration's loss for four positions: pure latency
        dict(name="loss_tiny", op="loss", n=4, V=4096, d=256, dtype="f32"),
        # perplexity of a short text on the 31B-shaped table: the table is streamed for 64 positions
        dict(name="loss_64", op="loss", n=64, V=262144, d=5376, dtype="bf16"),
        # odd sizes all round, half precision
        dict(name="loss_odd", op="loss", n=333, V=50001, d=1000, dtype="f16"),
        # the forward pass of a batch of 1,024 positions
        dict(name="loss_1024", op="loss", n=1024, V=262144, d=5120, dtype="bf16"),
        # the tiny configuration's gradients for four positions: pure latency
        dict(name="grad_tiny", op="grad", n=4, V=4096, d=256, dtype="f32", table=True, zloss=False),
        # gradients of 64 positions on the 31B-shaped table: the table read, its gradient written
        dict(name="grad_64", op="grad", n=64, V=262144, d=5376, dtype="bf16", table=True, zloss=False),
        # a frozen head under a trained body: the residual rows' gradient alone
        dict(name="grad_frozen_head", op="grad", n=2048, V=151936, d=896, dtype="bf16", table=False, zloss=True),
        # the backward pass of 4,096 positions: bound by the matrix cores
        dict(name="grad_4096", op="grad", n=4096, V=262144, d=5120, dtype="bf16", table=True, zloss=False),
        # loss, gradients and the gather's gradient into the same tied table
        dict(name="step_tied", op="step", n=1000, V=151936, d=896, dtype="bf16", zloss=True),
        # the gather's gradient of one long prompt with few distinct tokens
        dict(name="rows_prompt", op="rows", n=628, V=151936, d=896, dtype="bf16", grad="f32", ids="few"),
        # the gather's gradient of 32 sequences of 512 tokens
        dict(name="rows_batch", op="rows", n=16384, V=262144, d=768, dtype="f32", grad="f32", ids="zipf"),
        # a large batch of half-width gradients into the 31B-shaped table
        dict(name="rows_large", op="rows", n=65536, V=262144, d=5376, dtype="bf16", grad="bf16", ids="zipf"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["loss", "loss", "grad", "grad", "step", "rows", "rows"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    if op == "rows":
        V, d = _log_int(rng, 1000, 262144), 8 * _log_int(rng, 8, 672)
        return dict(op=op, n=_log_int(rng, 1, 65536), V=V, d=d, dtype=dtype,
                    grad=rng.choice(["f32", "f32", dtype]), ids=rng.choice(["zipf", "zipf", "few", "uniform"]))
    if dtype == "f32":  # full-precision tables are small ones
        n, V, d = _log_int(rng, 1, 1024), _log_int(rng, 1000, 32768), 4 * _log_int(rng, 16, 256)
    else:
        n, V, d = _log_int(rng, 1, 4096), _log_int(rng, 1000, 262144), 8 * _log_int(rng, 8, 640)
    case = dict(op=op, n=n, V=V, d=d, dtype=dtype)
    if op == "grad":
        case["table"] = rng.random() < 0.7
    if op != "loss":
        case["zloss"] = rng.random() < 0.3
    return case


def _ids(g, n, V, kind):
    """Token ids: uniform, Zipf(1.1) over the vocabulary, or Zipf over 109 distinct ones."""
    if kind == "uniform":
        return torch.randint(V, (n,), generator=g, device="cuda", dtype=torch.int32)
    top = min(109, V) if kind == "few" else V
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = (u * (float(top + 1) ** -0.1 - 1.0) + 1.0).pow(-10.0).floor().clamp_(1, top).to(torch.int64) - 1
    step = V // 2 + 1  # spreads the ranks over the table's rows
    while _gcd(step, V) != 1:
        step += 1
    return (rank * step % V).to(torch.int32)


def _gcd(a, b):
    while b:
        a, b = b, a % b
    return a


def _normal(g, rows, cols, dtype, size):
    x = torch.empty((rows, cols), dtype=dtype, device="cuda")
    step = max(1, (1 << 28) // cols)
    for r in range(0, rows, step):
        part = torch.randn((min(step, rows - r), cols), generator=g, device="cuda", dtype=torch.float32)
        x[r:r + step] = part.mul_(size).to(dtype)
    return x


def _log_partition(x, E):
    """ln sum_v exp(x . E_v) of every row, f32, by pieces of the vocabulary."""
    total = None
    for v in range(0, E.shape[0], 32768):
        part = torch.logsumexp(x.float() @ E[v:v + 32768].float().t(), 1, keepdim=False).double()
        total = part if total is None else torch.logaddexp(total, part)
    return total.float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, n, V, d, dtype = case["op"], case["n"], case["V"], case["d"], DTYPES[case["dtype"]]
    if op == "rows":
        # the table itself takes no part in its gradient; a few ids are bad ones (padding of -1)
        ids = _ids(g, n, V, case["ids"])
        ids = torch.where(torch.rand(n, generator=g, device="cuda") < 0.02, torch.full_like(ids, -1), ids)
        return dict(case=case, E=torch.zeros((V, d), dtype=dtype, device="cuda"), ids=ids, scale=float(d) ** 0.5,
                    grad=_normal(g, n, d, DTYPES[case["grad"]], 0.01))
    # residual rows of a partly trained model: the target stands out by nothing to about 17 nats
    E = _normal(g, V, d, dtype, 0.02)
    labels = _ids(g, n, V, "zipf")
    lift = torch.rand((n, 1), generator=g, device="cuda") * 17.0
    target = E[labels.long()].float()
    x = torch.randn((n, d), generator=g, device="cuda") + target * (lift / target.square().sum(1, keepdim=True))
    x = x.to(dtype)
    # one position in 16 has no target (a prompt or padding)
    labels = torch.where(torch.rand(n, generator=g, device="cuda") < 1 / 16, torch.full_like(labels, -100), labels)
    state = dict(case=case, E=E, x=x, labels=labels)
    if op != "loss":
        count = (labels >= 0).sum().clamp(min=1).float()
        size = 4096.0 if dtype == torch.float16 else 1.0  # half precision is trained with a scaled loss
        # the mean over the positions with a target, and 1e-4 lse^2 averaged over all positions
        state["grad_loss"] = torch.full((n,), size, device="cuda") / count
        state["lse"] = _log_partition(x, E)
        state["grad_lse"] = (2e-4 * size / n) * state["lse"] if case["zloss"] else None
    if op == "step":
        state["ids"] = _ids(g, n, V, "zipf")
        state["scale"] = float(d) ** 0.5
        state["grad"] = _normal(g, n, d, torch.float32, 2e-4 * size)
    return state


def _plain_logits(s):
    return s["x"].float() @ s["E"].float().t()


def _plain_loss(s):
    logits = _plain_logits(s)
    top = logits.amax(1, keepdim=True)
    lse = top[:, 0] + (logits - top).exp_().sum(1).log()
    labels = s["labels"].long()
    valid = (labels >= 0) & (labels < logits.shape[1])
    target = logits.gather(1, torch.where(valid, labels, torch.zeros_like(labels))[:, None])[:, 0]
    return torch.where(valid, lse - target, torch.zeros_like(lse)), lse


def _plain_grad(s, table):
    """f32 gradients of the residual rows and of the table."""
    labels = s["labels"].long()
    valid = (labels >= 0) & (labels < s["E"].shape[0])
    gl = torch.where(valid, s["grad_loss"], torch.zeros_like(s["grad_loss"]))
    both = gl if s["grad_lse"] is None else gl + s["grad_lse"]
    D = (_plain_logits(s) - s["lse"][:, None]).exp_() * both[:, None]
    D.scatter_add_(1, torch.where(valid, labels, torch.zeros_like(labels))[:, None], -gl[:, None])
    return D @ s["E"].float(), D.t() @ s["x"].float() if table else None


def _plain_rows(s, into):
    ids = s["ids"].long()
    valid = (ids >= 0) & (ids < into.shape[0])
    part = torch.where(valid[:, None], s["grad"].float() * s["scale"], torch.zeros_like(s["grad"], dtype=torch.float32))
    return into.index_add_(0, torch.where(valid, ids, torch.zeros_like(ids)), part)


def run(state):
    s, op = state, state["case"]["op"]
    dtype = s["E"].dtype
    if own:
        import embedding_table_gather_amd as etg
        t = s.get("table")
        if t is None:  # the handle that a program keeps beside its table
            t = s["table"] = etg.Table(s["E"], {torch.float32: etg.F32, torch.bfloat16: etg.BF16,
                                                torch.float16: etg.F16}[dtype], *s["E"].shape)
        if op == "rows":
            return dict(d_table=t.embed_gather_grad(s["grad"], s["ids"], scale=s["scale"]))
        if op == "loss":
            loss, lse = t.cross_entropy(s["x"], s["labels"])
            return dict(loss=loss, lse=lse)
        if op == "grad":
            dx, dE = t.cross_entropy_grad(s["x"], s["labels"], s["lse"], s["grad_loss"], s["grad_lse"],
                                          table_grad=s["case"]["table"])
            return dict(d_residual=dx, d_table=dE)
        loss, lse = t.cross_entropy(s["x"], s["labels"])
        dx, dE = t.cross_entropy_grad(s["x"], s["labels"], lse, s["grad_loss"], s["grad_lse"])
        t.embed_gather_grad(s["grad"], s["ids"], scale=s["scale"], out=dE, accumulate=True)
        return dict(loss=loss, d_residual=dx, d_table=dE)
    if op == "rows":
        return dict(d_table=_plain_rows(s, torch.zeros(s["E"].shape, device="cuda")).to(dtype))
    if op == "loss":
        loss, lse = _plain_loss(s)
        return dict(loss=loss, lse=lse)
    if op == "grad":
        dx, dE = _plain_grad(s, s["case"]["table"])
        return dict(d_residual=dx.to(dtype), d_table=None if dE is None else dE.to(dtype))
    loss, lse = _plain_loss(s)
    dx, dE = _plain_grad(dict(s, lse=lse), True)
    return dict(loss=loss, d_residual=dx.to(dtype), d_table=_plain_rows(s, dE).to(dtype))


def work(case):
    """Three products where both gradients are asked for and two for the residual rows' alone: the
    logits, which are not kept, count once per call that needs them."""
    op, n, V, d, size = case["op"], case["n"], case["V"], case["d"], SIZES[case["dtype"]]
    if op == "rows":
        return dict(bytes=n * d * SIZES[case["grad"]] + 4 * n + V * d * size, flops=n * d)
    x, E = n * d * size, V * d * size
    if op == "loss":
        return dict(bytes=x + E + 12 * n, flops=2 * n * V * d)
    if op == "grad":
        return dict(bytes=2 * x + E + (E if case["table"] else 0) + 16 * n,
                    flops=(6 if case["table"] else 4) * n * V * d)
    return dict(bytes=2 * x + 2 * E + 20 * n + 4 * n * d, flops=6 * n * V * d)


def exact(case, seed):
    """In 64 bits, by pieces of the vocabulary (rows: a sum per distinct token over the sorted ids)."""
    s = prepare(case, seed)
    op, n, V, d = case["op"], case["n"], case["V"], case["d"]
    if op == "rows":
        return dict(d_table=_exact_rows(s, torch.zeros((V, d), dtype=torch.float64, device="cuda")))
    x = s["x"].double()
    pieces = [(v, min(v + 16384, V)) for v in range(0, V, 16384)]
    row = torch.arange(n, device="cuda")
    y = s["labels"].long()
    has = (y >= 0) & (y < V)
    if op != "grad":
        best = torch.full((n,), float("-inf"), dtype=torch.float64, device="cuda")
        total = torch.zeros(n, dtype=torch.float64, device="cuda")
        for a, b in pieces:
            part = torch.matmul(x, s["E"][a:b].double().t().contiguous())
            new = torch.maximum(best, part.max(1).values)
            total = total * torch.exp(best - new) + torch.exp(part - new[:, None]).sum(1)
            best = new
        lse = best + torch.log(total)
        at = (x * s["E"][y.clamp(0, V - 1)].double()).sum(1)
        loss = torch.where(has, lse - at, torch.zeros_like(at))
        if op == "loss":
            return dict(loss=loss, lse=lse)
    else:
        lse = s["lse"].double()
    want_table = op == "step" or case["table"]
    gl = s["grad_loss"].double() * has
    gz = s["grad_lse"].double() if s["grad_lse"] is not None else torch.zeros_like(gl)
    dx = torch.zeros((n, d), dtype=torch.float64, device="cuda")
    dE = torch.zeros((V, d), dtype=torch.float64, device="cuda") if want_table else None
    for a, b in pieces:
        rows = s["E"][a:b].double()
        D = torch.exp(torch.matmul(x, rows.t().contiguous()) - lse[:, None]) * (gl + gz)[:, None]
        here = has & (y >= a) & (y < b)
        D[row[here], y[here] - a] -= gl[here]
        dx += torch.matmul(D, rows)
        if want_table:
            dE[a:b] = torch.matmul(D.t().contiguous(), x)
    if op == "grad":
        return dict(d_residual=dx, d_table=dE)
    return dict(loss=loss, d_residual=dx, d_table=_exact_rows(s, dE))


def _exact_rows(s, into):
    """into += the gradient rows summed per token, from running sums over the rows sorted by token."""
    ids = s["ids"].long()
    keep = torch.nonzero((ids >= 0) & (ids < into.shape[0]))[:, 0]
    if keep.numel() == 0:
        return into
    order = keep[torch.sort(ids[keep], stable=True).indices]
    token, count = torch.unique_consecutive(ids[order], return_counts=True)
    last = torch.cumsum(count, 0) - 1
    for c in range(0, into.shape[1], 512):
        sums = torch.cumsum(s["grad"][order, c:c + 512].double(), 0)[last]
        sums[1:] -= sums[:-1].clone()
        into[token, c:c + 512] += sums * s["scale"]
    return into
