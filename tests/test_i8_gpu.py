"""Row quantisation to int8 and the int8 product on the GPU.

Both definitions fix every rounding (correctly rounded f32 quotients; an exact integer
sum, one rounding to f32, one per scale, one to the output type), so results are
compared bit for bit with a 64-bit numpy form: the tolerance is zero.
"""
import numpy as np
import pytest
import torch

import embedding_table_gather_amd as etg
import oracle
import synth
from tests import decode_oracle as do
from tests.gpu_util import bits, note, table, to_dev

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _host_values(t):
    return t.float().cpu().numpy()


def _check_quantized(codes, scale, x):
    want_q, want_s = do.quantize(_host_values(x))
    assert np.array_equal(scale.cpu().numpy(), want_s, equal_nan=True)
    got = codes.cpu().numpy()
    bad = np.argwhere(got != want_q)
    assert bad.size == 0, f"{len(bad)} codes differ, first at {bad[0].tolist()}"


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 5376), (3, 7), (5, 64), (2, 255), (4, 1001), (65, 896), (1000, 33),
                                       (7, 4099), (3, 16384), (2, 20000), (2, 65536)])
def test_quantize_bit_exact(dtype, rows, cols):
    note(f"quantize {dtype} {rows} x {cols}")
    x = torch.from_numpy(synth.residuals(rows, cols, seed=rows + cols)).to(DTYPES[dtype]).cuda()
    codes, scale = etg.quantize_i8(x)
    torch.cuda.synchronize()
    assert codes.shape == (rows, cols) and codes.dtype == torch.int8 and scale.shape == (rows,)
    _check_quantized(codes, scale, x)


@pytest.mark.parametrize("cols", [16, 77, 896, 9000])
def test_quantize_special_rows(cols):
    # all zero; one value; halves of a step on both sides (ties to even); the smallest
    # subnormals (scale 0 or a subnormal); the largest values; a NaN; infinities
    x = np.zeros((10, cols), np.float32)
    x[1, cols // 2] = -3.5
    x[2] = np.arange(cols) % 255 - 127
    x[2, 0] = 127.0
    x[3] = (np.arange(cols) % 254 - 126.5).astype(np.float32)
    x[3, cols - 1] = 127.0
    x[4] = np.float32(1e-45) * (np.arange(cols) % 5)
    x[5] = np.float32(1e-42) * (np.arange(cols) % 9 - 4)
    x[6] = np.float32(3.4028235e38) * np.where(np.arange(cols) % 2, 1, -1)
    x[7] = 1.0
    x[7, cols - 1] = np.nan
    x[8] = 1.0
    x[8, 0] = np.inf
    x[9] = np.random.default_rng(3).standard_normal(cols)
    x[9, 1] = -np.inf
    note(f"quantize special rows, {cols}")
    d = to_dev(x)
    codes, scale = etg.quantize_i8(d)
    torch.cuda.synchronize()
    _check_quantized(codes, scale, d)
    assert np.isnan(scale.cpu().numpy()[7:]).all() and not codes[7:].any()


@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_quantize_near_half_steps(dtype):
    # x / scale next to every half-integer: 127 * scale is the row's largest value, the
    # others are (j + 1/2) * scale and its neighbours in the input type
    t = DTYPES[dtype]
    rows = []
    for top in (127.0, 1.0, 3.3, 0.0117, 250.0):
        top = float(torch.tensor(top, dtype=t).float())
        s = np.float32(top) / np.float32(127)
        j = torch.tensor([(i + 0.5) * float(s) for i in range(-127, 127)], dtype=torch.float64).to(t)
        step = torch.tensor([1e-7, -1e-7, 3e-3, -3e-3, 0.0], dtype=torch.float64)
        vals = torch.cat([(j.double() * (1 + e)).to(t) for e in step] + [torch.tensor([top, -top], dtype=t)])
        rows.append(vals.clamp(-top, top))
    x = torch.stack(rows).cuda()
    note(f"quantize near half steps {dtype}")
    codes, scale = etg.quantize_i8(x)
    torch.cuda.synchronize()
    _check_quantized(codes, scale, x)


@pytest.mark.parametrize("dtype,cols,x_pad,q_pad,offset", [("f32", 100, 3, 5, 1), ("bf16", 257, 1, 0, 3),
                                                            ("f16", 64, 64, 16, 0), ("bf16", 512, 7, 9, 1)])
def test_quantize_strides_leave_the_rest(dtype, cols, x_pad, q_pad, offset):
    rows = 9
    buf = torch.randn(rows * (cols + x_pad) + offset, device="cuda").to(DTYPES[dtype])
    x = buf[offset:].view(rows, cols + x_pad)[:, :cols]
    q = torch.full((rows * (cols + q_pad) + offset,), 55, dtype=torch.int8, device="cuda")
    codes = q[offset:].view(rows, cols + q_pad)[:, :cols]
    sbuf = torch.full((rows, 3), -1.0, device="cuda")
    note(f"quantize strided {dtype} {cols}")
    etg.quantize_i8(x, codes=codes, scale=sbuf[:, 1])
    torch.cuda.synchronize()
    _check_quantized(codes, sbuf[:, 1], x)
    rest = q[offset:].view(rows, cols + q_pad)[:, cols:]
    assert (rest == 55).all() and (q[:offset] == 55).all() and (sbuf[:, 0] == -1).all() and (sbuf[:, 2] == -1).all()


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("rows,cols", [(3, 8191), (2, 16385), (1500, 16400), (3, 20001), (2, 65535)])
def test_quantize_long_rows(dtype, rows, cols):
    # rows past what stays in registers, the largest value and NaNs in any piece
    x = np.random.default_rng(cols).standard_normal((rows, cols)).astype(np.float32)
    x[0, cols - 1] = 40.0
    x[1, 1] = -40.0
    if rows > 2:
        x[2, cols - 2] = np.nan
    note(f"quantize long rows {dtype} {rows} x {cols}")
    d = torch.from_numpy(x).to(DTYPES[dtype]).cuda()
    codes, scale = etg.quantize_i8(d)
    torch.cuda.synchronize()
    _check_quantized(codes, scale, d)


def test_quantize_is_the_wire_encoding():
    V, d, n = 500, 896, 33
    host = synth.make_table(synth.BF16, V, d, seed=9)
    t = table(host, synth.BF16, V, d)
    ids = torch.from_numpy(synth.uniform_ids(n, V, seed=10)).cuda()
    wire = t.embed_gather_wire(ids, etg.WIRE_I8)
    codes, scale = etg.quantize_i8(t.embed_gather(ids))
    torch.cuda.synchronize()
    assert torch.equal(wire[:, 8:].view(torch.int8), codes)
    assert torch.equal(wire[:, :4].contiguous().view(torch.float32)[:, 0], scale)


def _codes(g, rows, cols):
    return g.integers(-128, 128, size=(rows, cols), dtype=np.int16).astype(np.int8)


def _out_bits(out):
    if out.dtype == torch.float32:
        return out.cpu().numpy().view(np.uint32)
    return out.view(torch.int16).cpu().numpy().view(np.uint16)


def _want_bits(x, dtype):
    if dtype == torch.float32:
        return x.view(np.uint32)
    if dtype == torch.bfloat16:
        return do.f32_to_bf16(x)
    with np.errstate(over="ignore"):
        return x.astype(np.float16).view(np.uint16)


def _check_product(out, a, sa, w, sw):
    got, want = _out_bits(out), _want_bits(do.product(a, sa, w, sw), out.dtype)
    bad = np.argwhere(got != want)
    assert bad.size == 0, f"{len(bad)} of {got.size} values differ, first at {bad[0].tolist()}"


SHAPES = [(1, 1, 1), (1, 17, 64), (1, 4096, 256), (2, 300, 5376), (3, 100, 33), (4, 2049, 1001), (8, 640, 768),
          (9, 515, 896), (16, 16, 64), (17, 65, 127), (33, 1000, 128), (48, 777, 5120), (64, 513, 256),
          (65, 1003, 896), (77, 501, 1001), (100, 2000, 65), (128, 128, 128), (129, 257, 4096), (200, 700, 320),
          (256, 1030, 512), (300, 600, 5376), (513, 771, 192), (1024, 300, 256), (1, 20000, 16), (5, 33, 65536)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_product_bit_exact(M, N, K, dtype):
    g = np.random.default_rng(M * 7 + N * 3 + K)
    a, w = _codes(g, M, K), _codes(g, N, K)
    sa = (g.random(M) * 0.01 + 1e-3).astype(np.float32)
    sw = (g.random(N) * 0.001 + 1e-4).astype(np.float32)
    note(f"product {M} x {N} x {K} -> {dtype}")
    out = etg.matmul_i8(to_dev(a), to_dev(sa), to_dev(w), to_dev(sw), out_dtype=DTYPES[dtype])
    torch.cuda.synchronize()
    assert out.shape == (M, N)
    _check_product(out, a, sa, w, sw)


# outputs of more tiles than the small products' kernel takes: streaming (up to 16 rows), passes
# of up to 192 rows, tiles of 256 rows; K of one step and of several, odd and even
LARGE = [(1, 40001, 77), (7, 33000, 1040), (16, 20003, 513), (17, 33000, 127), (33, 32900, 300), (40, 33001, 272),
         (64, 33001, 1001), (65, 17003, 896), (77, 20011, 1001), (96, 17000, 16), (100, 20011, 16), (128, 16500, 513),
         (129, 16411, 1001), (150, 12001, 256), (192, 11000, 896), (200, 8300, 1001), (129, 12001, 333),
         (256, 9001, 256), (300, 8200, 1040), (513, 5003, 192), (1024, 2200, 640), (5, 8300, 10500), (40, 16450, 10300)]


@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_large_product_bit_exact(M, N, K, dtype):
    test_product_bit_exact(M, N, K, dtype)


def test_product_rows_far_apart():
    # more than 2^22 bytes between the rows of w, past the 32-bit offsets of the block kernels
    M, N, K, apart = 200, 8300, 80, (1 << 22) + 272
    g = np.random.default_rng(12)
    a, w = _codes(g, M, K), _codes(g, N, K)
    sa, sw = g.random(M).astype(np.float32), g.random(N).astype(np.float32)
    big = torch.empty((N - 1) * apart + K, dtype=torch.int8, device="cuda")
    wv = torch.as_strided(big, (N, K), (apart, 1))
    wv.copy_(to_dev(w))
    note("product rows far apart")
    out = etg.matmul_i8(to_dev(a), to_dev(sa), wv, to_dev(sw))
    torch.cuda.synchronize()
    _check_product(out, a, sa, w, sw)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_product_extreme_codes_and_scales(M):
    # the largest sum, 65536 * 128 * 128 = 2^30; scales of zero, a subnormal, huge, NaN
    N, K = 40, 65536
    a = np.full((M, K), -128, np.int8)
    w = np.full((N, K), -128, np.int8)
    w[1::2] = 127
    a[0, ::3] = 127
    sa = np.full(M, 1.0, np.float32)
    sw = np.ones(N, np.float32)
    sw[:6] = [0.0, 1e-42, 1e30, np.nan, -2.0, 3e-39]
    sa[M // 2] = 1e20
    note(f"product extremes M={M}")
    for dtype in DTYPES.values():
        out = etg.matmul_i8(to_dev(a), to_dev(sa), to_dev(w), to_dev(sw), out_dtype=dtype)
        torch.cuda.synchronize()
        want = do.product(a, sa, w, sw)
        nan = np.isnan(want)
        assert np.array_equal(torch.isnan(out).cpu().numpy(), nan) and nan[:, 3].all()
        assert np.array_equal(_out_bits(out)[~nan], _want_bits(want, dtype)[~nan])


@pytest.mark.parametrize("M,N,K,pad,shift", [(1, 200, 100, 1, 0), (6, 333, 256, 16, 0), (6, 333, 256, 3, 5),
                                             (40, 150, 512, 8, 8), (70, 300, 320, 16, 0), (300, 290, 448, 4, 1),
                                             (300, 513, 448, 16, 16), (9, 20005, 144, 5, 3), (40, 33003, 144, 8, 8),
                                             (80, 20001, 400, 1, 2), (300, 8301, 272, 3, 1), (300, 8301, 272, 48, 16)])
def test_product_strides_leave_the_rest(M, N, K, pad, shift):
    g = np.random.default_rng(M + N + K)
    a, w = _codes(g, M, K), _codes(g, N, K)
    sa, sw = g.random(M).astype(np.float32), g.random(N).astype(np.float32)

    def strided(q):
        buf = torch.full((q.shape[0] * (K + pad) + shift + K,), -77, dtype=torch.int8, device="cuda")
        v = buf[shift:shift + q.shape[0] * (K + pad)].view(q.shape[0], K + pad)[:, :K]
        v.copy_(to_dev(q))
        return v

    out = torch.full((M, N + 5), -7.0, device="cuda")
    s2 = torch.zeros((N, 2), device="cuda")
    s2[:, 1] = to_dev(sw)
    note(f"product strided {M} x {N} x {K} pad {pad} shift {shift}")
    etg.matmul_i8(strided(a), to_dev(sa), strided(w), s2[:, 1], out=out[:, :N])
    torch.cuda.synchronize()
    _check_product(out[:, :N].contiguous(), a, sa, w, sw)
    assert (out[:, N:] == -7.0).all()
    out16 = torch.full((M, N + 3), -7.0, device="cuda", dtype=torch.bfloat16)
    etg.matmul_i8(strided(a), to_dev(sa), strided(w), s2[:, 1], out=out16[:, 1:N + 1])
    torch.cuda.synchronize()
    _check_product(out16[:, 1:N + 1].contiguous(), a, sa, w, sw)
    assert (out16[:, 0] == -7.0).all() and (out16[:, N + 1:] == -7.0).all()


@pytest.mark.parametrize("M", [20, 300])
def test_output_offsets_past_32_bits(M):
    # output rows far enough apart that the last begins past 2^32 bytes
    N, K = 33000 if M == 20 else 8300, 64
    g = np.random.default_rng(M)
    a, w = _codes(g, M, K), _codes(g, N, K)
    sa, sw = g.random(M).astype(np.float32), g.random(N).astype(np.float32)
    apart = (1 << 32) // (2 * (M - 1)) + 8
    big = torch.empty((M - 1) * apart + N, dtype=torch.bfloat16, device="cuda")
    out = torch.as_strided(big, (M, N), (apart, 1))
    note(f"output offsets past 32 bits M={M}")
    etg.matmul_i8(to_dev(a), to_dev(sa), to_dev(w), to_dev(sw), out=out)
    torch.cuda.synchronize()
    _check_product(out.contiguous(), a, sa, w, sw)


def test_product_offsets_past_32_bits():
    # rows of w, a and the output more than 2^32 bytes apart; only the rows are written
    M, N, K = 3, 3, 96
    g = np.random.default_rng(5)
    a, w = _codes(g, M, K), _codes(g, N, K)
    sa, sw = g.random(M).astype(np.float32), g.random(N).astype(np.float32)
    apart = (1 << 32) + 48
    big = torch.empty(2 * apart + 4096, dtype=torch.int8, device="cuda")
    av = torch.as_strided(big, (M, K), (apart, 1))
    wv = torch.as_strided(big, (N, K), (apart, 1), 1024)
    av.copy_(to_dev(a))
    wv.copy_(to_dev(w))
    out = torch.as_strided(big.view(torch.float32), (M, N), (apart // 4, 1), 512)
    note("product offsets past 32 bits")
    etg.matmul_i8(av, to_dev(sa), wv, to_dev(sw), out=out)
    q = torch.as_strided(big, (M, N), (apart, 1), 2560)
    codes, scale = etg.quantize_i8(out, codes=q)
    torch.cuda.synchronize()
    _check_product(out.contiguous(), a, sa, w, sw)
    _check_quantized(codes, scale, out)


@pytest.mark.parametrize("M,K", [(1, 8), (1, 16), (17, 32)])
def test_more_rows_of_w_than_one_launch_takes(M, K):
    # sums below 2^24: a float32 matrix product is exact, and scales of 1 leave one rounding
    N = (1 << 28) + 100
    w = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda")
    a = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda")
    one = torch.ones(1, device="cuda")
    sw = torch.ones(N, device="cuda")
    note(f"product {M} x {N} x {K}")
    out = etg.matmul_i8(a, one.repeat(M), w, sw, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    step = 1 << 24
    for n in range(0, N, step):
        want = torch.matmul(a.float(), w[n:n + step].float().t().contiguous())
        assert torch.equal(out[:, n:n + step], want.to(torch.bfloat16)), n


def test_empty_calls_write_nothing():
    e8 = torch.empty((0, 64), dtype=torch.int8, device="cuda")
    w = torch.ones((5, 64), dtype=torch.int8, device="cuda")
    s0, s5 = torch.empty(0, device="cuda"), torch.ones(5, device="cuda")
    assert etg.matmul_i8(e8, s0, w, s5).shape == (0, 5)
    assert etg.matmul_i8(w, s5, e8, s0).shape == (5, 0)
    codes, scale = etg.quantize_i8(torch.empty((0, 64), device="cuda"))
    assert codes.shape == (0, 64) and scale.shape == (0,)


@pytest.mark.parametrize("dtype", [synth.F32, synth.BF16, synth.F16])
def test_i8_table_logits(dtype):
    # the quantised table's logits are the product of the quantised rows, and stay near
    # the unquantised table's: |dL| <= sum_i (|r_i| de_i + |e_i| dr_i + dr_i de_i) with
    # dr, de at most half a step (1/2 + 2^-20 for the f32 quotients) of each row's scale
    V, d, B = 700, 512, 5
    host = synth.make_table(dtype, V, d, seed=21)
    t = table(host, dtype, V, d)
    R = synth.residuals(B, d, seed=22)
    q = t.quantize_i8()
    note(f"I8Table dtype={dtype}")
    got = q.logits_raw(to_dev(R))
    a, sa = do.quantize(R)
    rows = {synth.F32: lambda: host, synth.BF16: lambda: do.bf16_to_f32(host),
            synth.F16: lambda: host.view(np.float16).astype(np.float32)}[dtype]().reshape(V, d)
    w, sw = do.quantize(rows)
    _check_product(got, a, sa, w, sw)
    L, _ = oracle.logits(host, dtype, V, d, R)
    half = 0.5 + 2.0 ** -20
    dr, de = half * sa.astype(np.float64)[:, None], half * sw.astype(np.float64)[None, :]
    bound = np.abs(R).astype(np.float64).sum(1)[:, None] * de + np.abs(rows).astype(np.float64).sum(1)[None, :] * dr \
        + d * dr * de
    assert (np.abs(got.cpu().numpy() - L) <= bound * (1 + 1e-6) + 1e-6).all()
    wire = oracle.wire_encode(R, etg.WIRE_I8)
    assert np.array_equal(bits(q.logits_raw_wire(torch.from_numpy(wire).cuda())), bits(got))


@pytest.mark.parametrize("M,N,K", [(17, 70, 1), (1, 130, 15), (3, 129, 7), (33, 64, 15), (65, 1000, 9), (16, 16, 4)])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_short_rows_bit_exact(M, N, K, dtype):
    # rows without a whole 16-byte load, one byte apart as well
    g = np.random.default_rng(M + N + K)
    a, w = _codes(g, M, K), _codes(g, N, K)
    sa, sw = g.random(M).astype(np.float32), g.random(N).astype(np.float32)
    note(f"product of short rows {M} x {N} x {K} -> {dtype}")
    out = etg.matmul_i8(to_dev(a), to_dev(sa), to_dev(w), to_dev(sw), out_dtype=DTYPES[dtype])
    wide = torch.full((N, K + 1), -128, dtype=torch.int8, device="cuda")
    wide[:, 1:] = to_dev(w)
    again = etg.matmul_i8(to_dev(a), to_dev(sa), wide[:, 1:], to_dev(sw), out_dtype=DTYPES[dtype])
    torch.cuda.synchronize()
    _check_product(out, a, sa, w, sw)
    assert torch.equal(again, out)
