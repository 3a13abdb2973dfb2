"""Sampling on the GPU against a 64-bit numpy form.

Ids are whole numbers and have to be equal.  A probability is a 64-bit quotient rounded
to f32 (half a step, 2^-24 of it); the total it is divided by is a sum of weights in
fixed point, each off by at most half a unit, which at 2^b tokens is at most 2^(2 b - 64)
of the total: 2^-24 at the largest vocabulary.  The tolerance is their sum, 2^-23, of the
value.
"""
import numpy as np
import pytest
import torch

import embedding_table_gather_amd as etg
import synth
from tests import decode_oracle as do
from tests.gpu_util import note, table, to_dev

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LAST_U = float(np.nextafter(np.float32(1), np.float32(0)))


def _per_row(v, rows):
    return v.cpu().numpy().tolist() if isinstance(v, torch.Tensor) else [v] * rows


def _want(logits, u, allowed, kw):
    l, u = logits.float().cpu().numpy(), u.cpu().numpy()
    rows = l.shape[0]
    cols = {k: _per_row(v, rows) for k, v in kw.items()}
    got = [do.sample_row(l[r], u[r], allowed=None if allowed is None else allowed[r if allowed.ndim == 2 else slice(None)],
                         **{k: c[r] for k, c in cols.items()}) for r in range(rows)]
    return np.array([g[0] for g in got], np.int32), np.array([g[1] for g in got])


def _check(logits, u, allowed=None, **kw):
    packed = None if allowed is None else torch.from_numpy(do.pack_allowed(allowed)).cuda()
    ids, probs = etg.sample(logits, u, allowed=packed, **kw)
    torch.cuda.synchronize()
    want_id, want_p = _want(logits, u, allowed, kw)
    got_id, got_p = ids.cpu().numpy(), probs.cpu().numpy().astype(np.float64)
    bad = np.flatnonzero(got_id != want_id)
    assert bad.size == 0, f"row {bad[0]}: {got_id[bad[0]]} instead of {want_id[bad[0]]} ({bad.size} rows differ)"
    assert (np.abs(got_p - want_p) <= 2.0 ** -23 * want_p).all(), (got_p, want_p)
    return ids, probs


def _logits(rows, V, dtype, seed, spread=2.5):
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, V), dtype=np.float32) * np.float32(spread)
    peaks = g.integers(0, V, size=(rows, min(V, 30)))
    np.put_along_axis(x, peaks, np.take_along_axis(x, peaks, 1)
                      + (g.random(peaks.shape) ** 2 * 5 * spread).astype(np.float32), 1)
    u = g.random(rows, dtype=np.float32)
    return torch.from_numpy(x).to(DTYPES[dtype]).cuda(), torch.from_numpy(u).cuda()


SETTINGS = [dict(), dict(temperature=0.0), dict(temperature=0.7, top_k=50), dict(top_k=1), dict(temperature=1.3, top_p=0.9),
            dict(min_p=0.05), dict(temperature=0.8, top_k=40, top_p=0.95, min_p=0.02), dict(temperature=0.1, top_k=300),
            dict(temperature=5.0, top_p=0.999), dict(top_p=1e-6), dict(min_p=1.0), dict(top_k=10 ** 9, top_p=0.5),
            dict(temperature=1e-30, top_p=0.5), dict(temperature=1e30, top_k=7), dict(temperature=3.0, top_k=2000)]


@pytest.mark.parametrize("how", range(len(SETTINGS)))
@pytest.mark.parametrize("rows,V,dtype", [(1, 1, "f32"), (3, 2, "bf16"), (2, 31, "f16"), (4, 64, "f32"), (3, 65, "bf16"),
                                          (5, 1000, "f32"), (3, 4097, "f16"), (2, 32003, "bf16"), (2, 151936, "f32")])
def test_sizes_and_settings(rows, V, dtype, how):
    note(f"sample {rows} x {V} {dtype} {SETTINGS[how]}")
    logits, u = _logits(rows, V, dtype, seed=V + how)
    _check(logits, u, **SETTINGS[how])


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("V", [50, 5000, 262144])
def test_settings_per_row(dtype, V):
    rows = 24
    logits, u = _logits(rows, V, dtype, seed=V)
    g = np.random.default_rng(V)
    u[0], u[1] = 0.0, LAST_U

    def pick(vals, t):
        return torch.tensor(g.choice(vals, rows).tolist(), dtype=t, device="cuda")
    note(f"sample per-row settings {dtype} V={V}")
    _check(logits, u, temperature=pick([0.0, 0.2, 0.7, 1.0, 1.5], torch.float32), top_k=pick([0, 1, 5, 50, 1000], torch.int32),
           top_p=pick([1.0, 0.3, 0.9, 0.99], torch.float32), min_p=pick([0.0, 0.01, 0.2], torch.float32))


@pytest.mark.parametrize("V", [7, 300, 20000])
def test_equal_logits_go_by_id(V):
    # all equal; two values; a few values many times over: the cut falls inside a tie
    g = np.random.default_rng(V)
    x = np.stack([np.full(V, 1.25), np.where(np.arange(V) % 3 == 1, 2.0, -1.0), g.integers(0, 4, V) * 0.5,
                  np.where(g.random(V) < 0.5, 0.0, -0.0), np.full(V, -3.4028235e38)]).astype(np.float32)
    for how in (dict(), dict(top_k=2), dict(top_k=V // 2 + 1), dict(top_p=0.5), dict(top_k=V // 2 + 1, top_p=0.75),
                dict(min_p=0.3), dict(top_p=0.25, min_p=0.5), dict(temperature=0.0)):
        for u in (0.0, 0.37, 0.5, LAST_U):
            note(f"sample ties V={V} {how} u={u}")
            _check(to_dev(x), torch.full((5,), u, device="cuda"), **how)


def test_infinities_nan_and_lowest_values():
    V = 1500
    g = np.random.default_rng(4)
    x = (g.standard_normal((10, V)) * 2).astype(np.float32)
    x[0, ::2] = -np.inf
    x[1] = -np.inf
    x[2] = np.nan
    x[3, 5::7] = np.nan
    x[4, [100, 900]] = np.inf                  # two infinite logits share all the mass
    x[5, 3:] = np.finfo(np.float32).min        # a mask of the type's lowest value
    x[6] = np.finfo(np.float32).min
    x[7, :] = -np.inf
    x[7, 1234] = -5.0
    x[8, :] = np.nan
    x[8, 77] = np.finfo(np.float32).max
    x[9, ::3] = -np.nan
    u = torch.from_numpy(g.random(10, dtype=np.float32)).cuda()
    for how in (dict(), dict(temperature=0.0), dict(temperature=0.6, top_k=30, top_p=0.9, min_p=0.01), dict(top_k=800),
                dict(top_p=0.999)):
        note(f"sample infinities {how}")
        ids, probs = _check(to_dev(x), u, **how)
        assert ids[1] == -1 and ids[2] == -1 and probs[1] == 0 and probs[2] == 0 and ids[7] == 1234


@pytest.mark.parametrize("dtype,V", [("f32", 33), ("bf16", 1000), ("f16", 32003)])
def test_allowed_masks(dtype, V):
    rows = 9
    logits, u = _logits(rows, V, dtype, seed=V)
    g = np.random.default_rng(V)
    mask = g.random((rows, V)) < np.array([1, 0, 0.5, 0.01, 0.9, 0.3, 0.1, 0.002, 0.5])[:, None]
    mask[2] = False
    mask[2, V - 1] = True
    for r in (0, 5):  # what is barred may hold anything
        barred = torch.from_numpy(~mask[r]).cuda()
        logits[r][barred] = float("nan") if r else float("inf")
    for how in (dict(), dict(temperature=0.0), dict(temperature=0.9, top_k=20, top_p=0.9)):
        note(f"sample masked {dtype} V={V} {how}")
        ids, _ = _check(logits, u, allowed=mask, **how)
        assert ids[1] == -1 and ids[2] == V - 1
    _check(logits, u, allowed=mask[4], top_p=0.8)  # one mask row for all


def test_settings_out_of_range_empty_the_row():
    rows, V = 12, 400
    logits, u = _logits(rows, V, "f32", seed=1)
    nan = float("nan")
    T = torch.tensor([1, -1, nan, float("inf"), 1, 1, 1, 1, 1, 1, 1, 1], dtype=torch.float32, device="cuda")
    k = torch.tensor([0, 0, 0, 0, -1, 0, 0, 0, 0, 0, 0, 5], dtype=torch.int32, device="cuda")
    p = torch.tensor([1, 1, 1, 1, 1, 0, 1.5, nan, 1, 1, 1, 1], dtype=torch.float32, device="cuda")
    mp = torch.tensor([0, 0, 0, 0, 0, 0, 0, 0, -0.5, 2, nan, 0], dtype=torch.float32, device="cuda")
    note("sample settings out of range")
    ids, _ = _check(logits, u, temperature=T, top_k=k, top_p=p, min_p=mp)
    assert (ids[1:11] == -1).all() and ids[0] >= 0 and ids[11] >= 0
    u = torch.tensor([0.5, 1.0, -0.1, nan, 2.0, 0.0] * 2, device="cuda")
    ids, _ = _check(logits, u)
    assert (ids[1:5] == -1).all() and ids[0] >= 0 and ids[5] >= 0


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("V,pad,offset", [(1000, 3, 1), (4096, 8, 0), (777, 0, 5)])
def test_strided_logits(dtype, V, pad, offset):
    rows = 4
    logits, u = _logits(rows, V, dtype, seed=V + pad)
    buf = torch.full((rows * (V + pad) + offset,), float("inf"), dtype=DTYPES[dtype], device="cuda")
    view = buf[offset:].view(rows, V + pad)[:, :V]
    view.copy_(logits)
    words = -(-V // 32)
    mask = np.random.default_rng(V).random((rows, V)) < 0.5
    wide = torch.full((rows, words + 2), -1, dtype=torch.int32, device="cuda")
    wide[:, :words] = torch.from_numpy(do.pack_allowed(mask)).cuda()
    note(f"sample strided {dtype} V={V} pad={pad}")
    _check(view, u, temperature=0.9, top_k=100, top_p=0.95)
    a, _ = etg.sample(view, u, allowed=wide[:, :words], top_k=30)
    b, _ = _check(logits, u, allowed=mask, top_k=30)
    assert torch.equal(a, b)


def test_offsets_past_32_bits():
    V, apart = 1000, (1 << 31) + 6
    big = torch.empty(2 * apart + V, dtype=torch.bfloat16, device="cuda")
    view = torch.as_strided(big, (3, V), (apart, 1))
    logits, u = _logits(3, V, "bf16", seed=8)
    view.copy_(logits)
    note("sample offsets past 32 bits")
    _check(view, u, top_k=60, top_p=0.9)


@pytest.mark.parametrize("V", [(1 << 19) + 3, 1 << 20])
def test_wide_vocabularies(V):
    g = torch.Generator(device="cuda").manual_seed(V)
    logits = torch.randn((2, V), generator=g, device="cuda") * 2
    u = torch.tensor([0.3, 0.9], device="cuda")
    note(f"sample V={V}")
    for how in (dict(), dict(top_k=100), dict(top_p=0.9), dict(top_p=0.999, min_p=1e-4)):
        _check(logits, u, **how)


@pytest.mark.parametrize("spread", [0.0, 1e-6, 0.01, 0.3, 30.0, 1e4, 1e30])
def test_logits_of_any_scale(spread):
    # nearly equal logits (every token in the nucleus) to ones that one token wins outright
    rows, V = 4, 30011
    logits, u = _logits(rows, V, "f32", seed=5, spread=spread)
    for how in (dict(), dict(top_k=1000), dict(top_p=0.7), dict(temperature=0.5, top_k=20000, top_p=0.9)):
        note(f"sample spread {spread} {how}")
        _check(logits, u, **how)


def test_more_flat_rows_than_histograms():
    # 3,600 rows that keep nearly all of their 2,100 tokens: more than the workspace has
    # histograms for, the rest go by passes over their logits
    rows, V = 3600, 2100
    logits, u = _logits(rows, V, "bf16", seed=6, spread=0.05)
    g = np.random.default_rng(6)

    def pick(vals, t):
        return torch.tensor(g.choice(vals, rows).tolist(), dtype=t, device="cuda")
    note("sample 3,600 flat rows")
    _check(logits, u, temperature=pick([0.5, 1.0], torch.float32), top_k=pick([0, 0, 2090], torch.int32),
           top_p=pick([1.0, 0.995, 0.999], torch.float32), min_p=pick([0.0, 0.01], torch.float32))


def test_large_batch_repeats_bitwise():
    rows, V = 300, 32003
    logits, u = _logits(rows, V, "bf16", seed=11, spread=1.5)
    note("sample 300 rows, twice")
    a = _check(logits, u, temperature=0.9, top_k=500, top_p=0.9)
    for _ in range(3):
        b = etg.sample(logits, u, temperature=0.9, top_k=500, top_p=0.9)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_draws_follow_the_distribution():
    # one row drawn at 4,096 evenly spaced random numbers: each kept token is drawn for
    # its share of them, to within one number at either end
    V, n = 500, 4096
    logits, _ = _logits(1, V, "f32", seed=2, spread=1.0)
    u = (torch.arange(n, device="cuda", dtype=torch.float32) + 0.5) / n
    ids, probs = etg.sample(logits.expand(n, V).contiguous(), u, top_k=40)
    torch.cuda.synchronize()
    got = np.bincount(ids.cpu().numpy(), minlength=V)
    p = np.zeros(V)
    p[ids.cpu().numpy()] = probs.cpu().numpy()
    assert np.abs(got - p * n).max() <= 1.0 + 1e-3
    assert (np.diff(ids.cpu().numpy()) >= 0).all()


def test_sample_empty_batch():
    ids, probs = etg.sample(torch.empty((0, 100), device="cuda"), torch.empty(0, device="cuda"))
    assert ids.shape == (0,) and probs.shape == (0,)


def _decode(t, q, ids, u):
    """Two steps of a decode loop on the quantised lm_head: gather, logits, next ids."""
    out = []
    for i in range(2):
        x = t.embed_gather(ids, scale="sqrt_d", check=False)
        ids, probs = q.sample(x, u[i], temperature=0.8, top_k=50, top_p=0.95, min_p=0.01)
        out += [ids, probs]
    return out


@pytest.mark.parametrize("V,d,B", [(5003, 896, 3), (4096, 256, 70)])
def test_decode_loop_of_all_operators(V, d, B):
    host = synth.make_table(synth.BF16, V, d, seed=31, std=0.05)
    t = table(host, synth.BF16, V, d)
    q = t.quantize_i8()
    ids = torch.from_numpy(synth.uniform_ids(B, V, seed=32)).cuda()
    u = torch.rand((2, B), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    note(f"decode loop V={V} d={d} B={B}")
    got = _decode(t, q, ids, u)
    torch.cuda.synchronize()
    rows = do.bf16_to_f32(host).reshape(V, d)
    w, sw = do.quantize(rows)
    cur = ids.cpu().numpy()
    for i in range(2):
        x = rows[cur] * np.float32(np.sqrt(np.float64(d)))
        a, sa = do.quantize(x)
        logits = do.product(a, sa, w, sw)
        want = [do.sample_row(logits[b], u[i, b].item(), 0.8, 50, 0.95, 0.01) for b in range(B)]
        cur = np.array([v[0] for v in want], np.int32)
        assert np.array_equal(got[2 * i].cpu().numpy(), cur)
        p = np.array([v[1] for v in want])
        assert (np.abs(got[2 * i + 1].cpu().numpy() - p) <= 2.0 ** -23 * p).all()
    # the unquantised table's own call gives what sample gives on its raw logits
    x = t.embed_gather(ids, scale="sqrt_d", check=False)
    a = t.sample(x, u[0], temperature=0.7, top_p=0.9)
    b = etg.sample(t.logits_raw(x), u[0], temperature=0.7, top_p=0.9)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_captured_loops_replay_on_two_streams():
    # two graphs of the same shapes, replayed at the same time: neither may write what the
    # other reads; each replay is checked against the eager call
    V, d, B = 5003, 512, 5
    t = table(synth.make_table(synth.BF16, V, d, seed=41, std=0.05), synth.BF16, V, d)
    q = t.quantize_i8()
    gen = torch.Generator(device="cuda").manual_seed(4)
    streams = [torch.cuda.Stream() for _ in range(2)]
    state = []
    for s in streams:
        ids = torch.randint(V, (B,), generator=gen, device="cuda", dtype=torch.int32)
        u = torch.rand((2, B), generator=gen, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            _decode(t, q, ids, u)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = _decode(t, q, ids, u)
        state.append((s, graph, ids, u, out))
    for turn in range(4):
        want = []
        for s, graph, ids, u, out in state:
            ids.copy_(torch.randint(V, (B,), generator=gen, device="cuda", dtype=torch.int32))
            u.copy_(torch.rand((2, B), generator=gen, device="cuda"))
            want.append([w.clone() for w in _decode(t, q, ids, u)])
        torch.cuda.synchronize()
        note(f"two graphs, replay {turn}")
        for s, graph, *_ in state:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (*_, out), w in zip(state, want):
            assert all(torch.equal(x, y) for x, y in zip(out, w))


def test_workspaces_and_settings_past_the_c_types():
    logits, u = _logits(2, 300, "f32", seed=3)
    want = etg.sample(logits, u)
    note("sample top_k 2^32 + 5")
    ids, probs = etg.sample(logits, u, top_k=2 ** 32 + 5)  # more than any vocabulary, not 5
    torch.cuda.synchronize()
    assert torch.equal(ids, want[0]) and torch.equal(probs, want[1])
    codes, scale = torch.zeros((2, 64), dtype=torch.int8, device="cuda"), torch.ones(2, device="cuda")
    head = etg.I8Table(codes, scale)
    for space in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 20, dtype=torch.float32, device="cuda"),
                  torch.empty(1 << 20, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            etg.sample(logits, u, workspace=space)
        with pytest.raises(ValueError, match="workspace"):
            etg.matmul_i8(codes, scale, codes, scale, workspace=space)
        with pytest.raises(ValueError, match="workspace"):
            head.logits_raw(torch.ones((1, 64), device="cuda"), workspace=space)


def test_calls_on_two_streams_at_once():
    V, d, B = 20011, 768, 16
    t = table(synth.make_table(synth.BF16, V, d, seed=51, std=0.05), synth.BF16, V, d)
    q = t.quantize_i8()
    gen = torch.Generator(device="cuda").manual_seed(5)
    xs = [torch.randn((B, d), generator=gen, device="cuda") for _ in range(2)]
    us = [torch.rand(B, generator=gen, device="cuda") for _ in range(2)]
    want = [q.sample(x, u, top_k=40, top_p=0.9) for x, u in zip(xs, us)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    note("two streams at once")
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(q.sample(xs[i], us[i], top_k=40, top_p=0.9))
    torch.cuda.synchronize()
    for i in range(2):
        for ids, probs in got[i]:
            assert torch.equal(ids, want[i][0]) and torch.equal(probs, want[i][1])


@pytest.mark.parametrize("dtype,view,nans", [("f32", torch.int32, (0x7F800001, -0x7FFFFF, 0x7FBFFFFF)),
                                             ("bf16", torch.int16, (0x7F81, -0x7F, 0x7FBF)),
                                             ("f16", torch.int16, (0x7C01, -0x3FF, 0x7DFF))])
@pytest.mark.parametrize("V", [8, 700, 20011])
def test_signaling_nan_logits(dtype, view, nans, V):
    # a signaling NaN at every place of a group of tokens after the row's largest logit, in the
    # first or the last group, alone or with one in every third place beside it
    logits, u = _logits(56, V, dtype, seed=V)
    bits = logits.view(view)
    pairs = [(a, b) for b in range(8) for a in range(b)]
    for r in range(56):
        first = 0 if r < 28 else V - 8
        a, b = pairs[r % 28]
        if r % 2:
            bits[r, 2::3] = nans[r % 3]
        logits[r, first + a] = 30.0
        bits[r, first + b] = nans[r % 3]
    for how in (dict(), dict(temperature=0.0), dict(temperature=2.0, top_k=40), dict(temperature=3.0, top_p=0.9),
                dict(temperature=4.0, min_p=0.01), dict(temperature=1e4, top_p=0.97)):
        note(f"sample signaling NaN {dtype} V={V} {how}")
        _check(logits, u, **how)


@pytest.mark.parametrize("V,spread", [(1, 1.0), (900, 2.5), (30011, 2.5), (30011, 0.01)])
def test_negative_zero_settings(V, spread):
    # -0 is 0: the first kept token for a random number, greedy for a temperature, off for min-p
    rows = 3
    logits, _ = _logits(rows, V, "f32", seed=V, spread=spread)
    zero = torch.zeros(rows, device="cuda")
    for how in (dict(), dict(temperature=0.7, top_k=20), dict(top_p=0.9), dict(min_p=0.01), dict(top_k=3000, top_p=0.8),
                dict(temperature=-0.0), dict(temperature=-zero), dict(min_p=-0.0, top_k=5), dict(min_p=-zero)):
        note(f"sample u = -0.0, V={V} spread={spread} {how}")
        got = _check(logits, -zero, **how)
        want = etg.sample(logits, zero, **how)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("k", [-1, -2 ** 31, -2 ** 31 - 1, -2 ** 32, -2 ** 32 + 5, -10 ** 30])
def test_negative_top_k_is_refused(k):
    logits, u = _logits(2, 300, "f32", seed=3)
    with pytest.raises(etg.EtgError, match="top_k") as e:
        etg.sample(logits, u, top_k=k)
    assert e.value.status == -5


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("V", [9000, 70001])
def test_top_tokens_side_by_side(dtype, V):
    # sorted logits, both ways, and a block of large ones: the first k lie in few groups of tokens,
    # all of whose other tokens are near them
    x = np.sort(np.random.default_rng(V).standard_normal((4, V), dtype=np.float32) * np.float32(2.5), axis=1)
    x[0] = x[0, ::-1]
    x[2] = np.roll(x[2], V // 3)
    x[3] = np.where((np.arange(V) > 4000) & (np.arange(V) < 8000), x[3] + 20, x[3])
    logits = torch.from_numpy(np.ascontiguousarray(x)).to(DTYPES[dtype]).cuda()
    u = torch.tensor([0.1, 0.5, 0.9, 0.999], device="cuda")
    for how in (dict(top_k=50), dict(top_k=1000, top_p=0.9), dict(temperature=0.5, top_k=700, min_p=0.3),
                dict(temperature=0.0), dict(top_p=0.6)):
        note(f"sample top tokens side by side {dtype} V={V} {how}")
        _check(logits, u, **how)
