"""Cases of the int8 lm_head and sampling operators: quantize_i8, matmul_i8, I8Table.logits_raw, sample.

Each case names one call of a serving loop.  ``run`` computes it either through this package
(``own`` true) or in a plain form of elementary torch operations (``own`` false).
"""
import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    """The shapes are this package's own configurations (262,144 x 5,376 and x 5,120, 151,936 and
    4,096 tokens) and generic odd ones."""
    return [
        # one residual row on its way to the int8 lm_head: pure latency
        dict(name="quantize_row", op="quantize", rows=1, cols=5376, dtype="f32"),
        # the residual rows of a large batch
        dict(name="quantize_batch", op="quantize", rows=1024, cols=5120, dtype="f32"),
        # a whole bf16 table turned into an int8 one, once per model load
        dict(name="quantize_table", op="quantize", rows=262144, cols=5376, dtype="bf16"),
        # the tiny configuration's lm_head for four residual rows
        dict(name="head_tiny", op="head", m=4, n=4096, k=256, out="f32"),
        # a decode step of one sequence: the whole int8 table is streamed for one row
        dict(name="head_decode_1", op="head", m=1, n=262144, k=5376, out="f32"),
        # a decode step of 64 sequences
        dict(name="head_decode_64", op="head", m=64, n=262144, k=5376, out="f32"),
        # odd sizes all round: rows of neither operand are aligned
        dict(name="product_odd", op="product", m=77, n=50001, k=1001, out="f16"),
        # scoring 1,024 positions against the whole vocabulary: bound by the matrix cores
        dict(name="product_batch", op="product", m=1024, n=262144, k=5120, out="bf16"),
        # the next token of one sequence
        dict(name="sample_1", op="sample", rows=1, vocab=262144, dtype="f32", params="one", mask=False, spread=2.5),
        # 64 sequences whose requests bring their own settings
        dict(name="sample_64", op="sample", rows=64, vocab=262144, dtype="f32", params="mixed", mask=False, spread=2.5),
        # a large batch on half-width logits
        dict(name="sample_1024", op="sample", rows=1024, vocab=151936, dtype="bf16", params="mixed", mask=False,
             spread=2.5),
        # decoding under a grammar: most tokens barred, one row with nothing left
        dict(name="sample_masked", op="sample", rows=33, vocab=32003, dtype="f16", params="mixed", mask=True,
             spread=1.5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "head", "sample", "sample"])
    if op == "quantize":
        rows, cols = _log_int(rng, 1, 262144), _log_int(rng, 1, 5376)
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(sorted(DTYPES)))
    if op in ("product", "head"):
        m, n, k = _log_int(rng, 1, 1024), _log_int(rng, 1, 262144), _log_int(rng, 1, 5120)
        if op == "head" or rng.random() < 0.5:
            k = -(-k // 32) * 32
        return dict(op=op, m=m, n=n, k=k, out=rng.choice(sorted(DTYPES)))
    vocab = _log_int(rng, 1, 262144)
    rows = min(_log_int(rng, 1, 1024), max(1, 1024 * 151936 // vocab))
    return dict(op=op, rows=rows, vocab=vocab, dtype=rng.choice(sorted(DTYPES)), params=rng.choice(["one", "mixed"]),
                mask=rng.random() < 0.3, spread=rng.choice([0.5, 1.5, 2.5, 4.0]))


def _codes(g, rows, cols):
    """int8 codes as quantising Gaussian rows gives them: largest magnitude 127 in about every row."""
    q = torch.empty((rows, cols), dtype=torch.int8, device="cuda")
    step = max(1, (1 << 28) // cols)
    for r in range(0, rows, step):
        part = torch.randn((min(step, rows - r), cols), generator=g, device="cuda", dtype=torch.float32)
        q[r:r + step] = part.mul_(34.0).round_().clamp_(-127, 127).to(torch.int8)
    return q


def _scales(g, rows, mean):
    return mean * (0.8 + 0.4 * torch.rand(rows, generator=g, device="cuda", dtype=torch.float32))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    if op == "quantize":
        dtype = DTYPES[case["dtype"]]
        x = torch.empty((case["rows"], case["cols"]), dtype=dtype, device="cuda")
        step = max(1, (1 << 28) // case["cols"])
        for r in range(0, case["rows"], step):  # table rows or residual rows of differing magnitudes
            part = torch.randn((min(step, case["rows"] - r), case["cols"]), generator=g, device="cuda")
            x[r:r + step] = (part * _scales(g, part.shape[0], 0.5)[:, None]).to(dtype)
        return dict(case=case, x=x)
    if op == "head":
        x = torch.randn((case["m"], case["k"]), generator=g, device="cuda")
        return dict(case=case, x=x, w=_codes(g, case["n"], case["k"]), w_scale=_scales(g, case["n"], 6e-4))
    if op == "product":
        return dict(case=case, a=_codes(g, case["m"], case["k"]), a_scale=_scales(g, case["m"], 0.03),
                    w=_codes(g, case["n"], case["k"]), w_scale=_scales(g, case["n"], 6e-4))
    rows, vocab = case["rows"], case["vocab"]
    logits = torch.empty((rows, vocab), dtype=DTYPES[case["dtype"]], device="cuda")
    peaks = min(vocab, 40)
    for r in range(0, rows, 64):  # a Gaussian bulk and a few dozen tokens that stand out of it
        part = torch.randn((min(64, rows - r), vocab), generator=g, device="cuda") * case["spread"]
        at = torch.randint(vocab, (part.shape[0], peaks), generator=g, device="cuda")
        lift = torch.rand((part.shape[0], peaks), generator=g, device="cuda").pow(2) * (6.0 * case["spread"])
        part.scatter_add_(1, at, lift)
        logits[r:r + 64] = part.to(logits.dtype)
    state = dict(case=case, logits=logits, uniform=torch.rand(rows, generator=g, device="cuda"), allowed=None)
    if case["params"] == "mixed":  # each request has its own settings, some of them switched off
        def pick(values, dtype):
            at = torch.randint(len(values), (rows,), generator=g, device="cuda")
            return torch.tensor(values, dtype=dtype, device="cuda")[at]
        state.update(temperature=pick([0.0, 0.3, 0.7, 0.8, 1.0, 1.5], torch.float32),
                     top_k=pick([0, 0, 1, 20, 50, 1000], torch.int32),
                     top_p=pick([1.0, 0.5, 0.9, 0.95, 0.99], torch.float32),
                     min_p=pick([0.0, 0.0, 0.02, 0.1], torch.float32))
    else:
        state.update(temperature=0.8, top_k=50, top_p=0.95, min_p=0.02)
    if case["mask"]:  # a bit per token, 1 = allowed; a grammar leaves a few or many, in one row none
        words = -(-vocab // 32)
        share = torch.rand((rows, 1, 1), generator=g, device="cuda").pow(4)
        if rows > 3:
            share[3] = 0.0
        bits = torch.rand((rows, words, 32), generator=g, device="cuda") < share
        weight = (1 << torch.arange(32, device="cuda", dtype=torch.int64))
        packed = (bits.to(torch.int64) * weight).sum(2)
        state["allowed"] = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)
    return state


def _plain_quantize(x):
    x = x.float()
    top = x.abs().amax(1)
    fine = torch.isfinite(top)
    scale = top / torch.full_like(top, 127.0)
    q = (x / scale[:, None]).round_().clamp_(-127.0, 127.0)
    q = torch.where((fine & (scale > 0))[:, None], q, torch.zeros_like(q)).to(torch.int8)
    return q, torch.where(fine, scale, torch.full_like(scale, float("nan")))


def _plain_product(a, a_scale, w, w_scale, dtype):
    sums = a.float() @ w.float().t()
    return (sums * a_scale[:, None] * w_scale[None, :]).to(dtype)


def _column(v, like, dtype):
    v = v if torch.is_tensor(v) else torch.full((like.shape[0],), v, device=like.device)
    return v.to(dtype)[:, None]


def _allowed_tokens(words, rows, vocab):
    at = torch.arange(vocab, device=words.device)
    return (words.expand(rows, -1)[:, at // 32] >> (at % 32).to(torch.int32)) & 1 != 0


def _plain_sample(s):
    """In 64 bits: an id changes where a running sum next to u * total is rounded."""
    l = s["logits"].double()
    rows, vocab = l.shape
    live = l > float("-inf")  # neither -inf nor NaN
    if s["allowed"] is not None:
        live &= _allowed_tokens(s["allowed"], rows, vocab)
    l = torch.where(live, l, torch.full_like(l, float("-inf")))
    temperature, top_k = _column(s["temperature"], l, torch.float64), _column(s["top_k"], l, torch.int64)
    top_p, min_p = _column(s["top_p"], l, torch.float64), _column(s["min_p"], l, torch.float64)
    sorted_l, order = torch.sort(l, dim=1, descending=True, stable=True)
    first = sorted_l[:, :1]
    place = torch.arange(vocab, device=l.device)[None, :]
    w = torch.exp((sorted_l - first) / temperature)
    w = torch.where((sorted_l == first) & (first > float("-inf")), torch.ones_like(w), w)
    w = torch.where(sorted_l > float("-inf"), w, torch.zeros_like(w))
    greedy = temperature == 0
    w = torch.where(greedy, ((place == 0) & (first > float("-inf"))).double(), w)
    kept = (top_k == 0) | (place < top_k)
    before = torch.cumsum(torch.where(kept, w, torch.zeros_like(w)), 1)
    mass = before[:, -1:].clone()
    before = torch.cat([torch.zeros_like(mass), before[:, :-1]], 1)
    kept &= (top_p >= 1) | (before < top_p * mass)
    kept &= w >= min_p
    w = torch.where(kept, w, torch.zeros_like(w))
    by_id = torch.zeros_like(w).scatter_(1, order, w)
    run_sum = torch.cumsum(by_id, 1)
    total = run_sum[:, -1:]
    ids = (run_sum <= s["uniform"].double()[:, None] * total).sum(1).clamp_(max=vocab - 1)
    prob = by_id.gather(1, ids[:, None])[:, 0] / total[:, 0]
    some = total[:, 0] > 0
    ids = torch.where(some, ids, torch.full_like(ids, -1)).to(torch.int32)
    return ids, torch.where(some, prob, torch.zeros_like(prob)).float()


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import embedding_table_gather_amd as etg
        if op == "quantize":
            codes, scale = etg.quantize_i8(state["x"])
            return dict(codes=codes, scale=scale)
        if op == "head":
            table = etg.I8Table(state["w"], state["w_scale"])
            return dict(logits=table.logits_raw(state["x"], out_dtype=DTYPES[case["out"]]))
        if op == "product":
            return dict(out=etg.matmul_i8(state["a"], state["a_scale"], state["w"], state["w_scale"],
                                          out_dtype=DTYPES[case["out"]]))
        ids, probs = etg.sample(state["logits"], state["uniform"], temperature=state["temperature"],
                                top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"],
                                allowed=state["allowed"])
        return dict(ids=ids, probs=probs)
    if op == "quantize":
        codes, scale = _plain_quantize(state["x"])
        return dict(codes=codes, scale=scale)
    if op == "head":
        codes, scale = _plain_quantize(state["x"])
        return dict(logits=_plain_product(codes, scale, state["w"], state["w_scale"], DTYPES[case["out"]]))
    if op == "product":
        return dict(out=_plain_product(state["a"], state["a_scale"], state["w"], state["w_scale"],
                                       DTYPES[case["out"]]))
    ids, probs = _plain_sample(state)
    return dict(ids=ids, probs=probs)


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return dict(bytes=n * (SIZES[case["dtype"]] + 1) + 4 * case["rows"], flops=3 * n)
    if op in ("product", "head"):
        m, n, k = case["m"], case["n"], case["k"]
        a = 4 * m * k if op == "head" else m * k + 4 * m
        return dict(bytes=a + n * k + 4 * n + m * n * SIZES[case["out"]], flops=2 * m * n * k)
    n = case["rows"] * case["vocab"]
    mask = case["rows"] * 4 * -(-case["vocab"] // 32) if case["mask"] else 0
    return dict(bytes=n * SIZES[case["dtype"]] + mask + 12 * case["rows"], flops=4 * n)


def _exact_codes(x):
    """scale and x / scale rounded to 32 bits from 64: the nearest 32-bit values of the quotients."""
    top = x.double().abs().max(1).values
    scale = (top / 127).float()
    q = torch.zeros(x.shape, dtype=torch.int8, device=x.device)
    for r in range(0, x.shape[0], 16384):
        s = scale[r:r + 16384, None].double()
        ratio = torch.where(s > 0, x[r:r + 16384].double() / s, torch.zeros_like(s)).float()
        q[r:r + 16384] = torch.round(ratio.double()).clamp(-127, 127).to(torch.int8)
    return q, scale, top / 127


def _exact_product(a, a_scale, w, w_scale):
    out = torch.empty((a.shape[0], w.shape[0]), dtype=torch.float64, device="cuda")
    ad, sd = a.double(), a_scale.double()[:, None]
    for n in range(0, w.shape[0], 16384):
        out[:, n:n + 16384] = torch.matmul(ad, w[n:n + 16384].double().t().contiguous()) * sd * \
            w_scale[n:n + 16384].double()[None, :]
    return out


def _exact_row(l, u, temperature, top_k, top_p, min_p):
    """(id, prob) of one row's candidates: their logits in 64 bits by id, -inf where there is none."""
    value, at = torch.sort(l, descending=True, stable=True)
    n = int((value > float("-inf")).sum())
    if n == 0:
        return -1, 0.0
    if temperature == 0:
        return int(at[0]), 1.0
    w = torch.where(value[:n] == value[0], 0.0, (value[:n] - value[0]) / temperature).exp()
    n = min(n, top_k) if top_k > 0 else n
    sums = torch.cumsum(w[:n], 0)
    if top_p < 1:
        n = min(n, int((sums < top_p * sums[-1]).sum()) + 1)
    n = min(n, int((w >= min_p).sum()))
    ids, back = torch.sort(at[:n])
    w = w[:n][back]
    sums = torch.cumsum(w, 0)
    j = min(int((sums <= u * sums[-1]).sum()), n - 1)
    return int(ids[j]), float(w[j] / sums[-1])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        codes, _, scale = _exact_codes(s["x"])
        return dict(codes=codes, scale=scale)
    if op == "head":
        codes, scale, _ = _exact_codes(s["x"])
        return dict(logits=_exact_product(codes, scale, s["w"], s["w_scale"]))
    if op == "product":
        return dict(out=_exact_product(s["a"], s["a_scale"], s["w"], s["w_scale"]))
    rows, vocab = s["logits"].shape
    column = {}
    for name in ("temperature", "top_k", "top_p", "min_p", "uniform"):
        v = s[name]
        column[name] = v.tolist() if torch.is_tensor(v) else [float(np.float32(v)) if name != "top_k" else v] * rows
    ids, probs = [], []
    for r in range(rows):
        l = s["logits"][r].double()
        live = ~torch.isnan(l)
        if s["allowed"] is not None:
            words = s["allowed"][r].cpu().numpy().view(np.uint8)
            live &= torch.from_numpy(np.unpackbits(words, bitorder="little")[:vocab] != 0).cuda()
        l = torch.where(live, l, torch.full_like(l, float("-inf")))
        i, p = _exact_row(l, column["uniform"][r], column["temperature"][r], column["top_k"][r], column["top_p"][r],
                          column["min_p"][r])
        ids.append(i)
        probs.append(p)
    return dict(ids=torch.tensor(ids, dtype=torch.int32), probs=torch.tensor(probs, dtype=torch.float64))
