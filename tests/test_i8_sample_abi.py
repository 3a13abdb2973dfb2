"""Refusals of the int8 lm_head and sampling entry points, on the host: nothing is launched."""
import ctypes

import pytest
import torch

import embedding_table_gather_amd as etg

FAKE = 0x10000  # an aligned address that is never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    return etg.lib()


def _err(L):
    return L.etg_last_error().decode()


def _p(off=0):
    return ctypes.c_void_p(FAKE + off)


def test_quantize_errors(L):
    f = L.etg_quantize_i8

    def call(x=_p(), dt=etg.F32, rows=4, cols=64, xs=64, q=_p(), qs=64, s=_p(), ss=1):
        return f(x, dt, rows, cols, xs, q, qs, s, ss, None)
    assert call(dt=etg.Q8_0) == -2 and "dtype" in _err(L)
    assert call(dt=9) == -2
    assert call(rows=-1) == -3 and call(rows=2 ** 31) == -3
    assert call(cols=0) == -3 and call(cols=65537, xs=65537, qs=65537) == -3 and "cols" in _err(L)
    assert call(xs=63) == -3 and "input stride" in _err(L)
    assert call(xs=2 ** 41) == -3
    assert call(qs=63) == -3 and "code stride" in _err(L)
    assert call(ss=0) == -3 and "scale stride" in _err(L)
    assert call(x=None) == -1 and call(q=None) == -1 and call(s=None) == -1
    assert call(x=_p(2)) == -4 and call(dt=etg.BF16, x=_p(1)) == -4 and call(s=_p(2)) == -4
    assert call(rows=0, x=None, q=None, s=None) == 0


def test_matmul_errors(L):
    f = L.etg_matmul_i8

    def call(a=_p(), as_=64, sa=_p(), sas=1, w=_p(), ws=64, sw=_p(), sws=1, m=4, n=100, k=64, out=_p(), dt=etg.F32,
             os_=100, work=_p(), nbytes=1 << 40):
        return f(a, as_, sa, sas, w, ws, sw, sws, m, n, k, out, dt, os_, work, nbytes, None)
    assert call(dt=etg.Q8_0) == -2 and "output dtype" in _err(L)
    assert call(m=-1) == -3 and call(m=65537) == -3 and "m " in _err(L)
    assert call(n=-1) == -3 and call(n=2 ** 31) == -3
    assert call(k=0) == -3 and call(k=65537) == -3 and "k " in _err(L)
    assert call(as_=63) == -3 and "a stride" in _err(L)
    assert call(ws=63) == -3 and "w stride" in _err(L)
    assert call(sas=0) == -3 and call(sws=-1) == -3
    assert call(os_=99) == -3 and "output stride" in _err(L)
    for name in ("a", "sa", "w", "sw", "out"):
        assert call(**{name: None}) == -1, name
    assert call(sa=_p(2)) == -4 and call(sw=_p(1)) == -4 and call(out=_p(2)) == -4
    assert call(dt=etg.F16, out=_p(1)) == -4
    need = L.etg_matmul_i8_workspace(4, 100, 64)
    assert need >= 0
    if need:
        assert call(work=None) == -1 and call(work=_p(16)) == -4
        assert call(nbytes=need - 1) == -6 and "workspace" in _err(L)
    assert call(m=0, a=None, out=None) == 0 and call(n=0, w=None, out=None) == 0
    assert L.etg_matmul_i8_workspace(65537, 1, 1) == -3 and L.etg_matmul_i8_workspace(1, 1, 0) == -3


def test_logits_i8_errors(L):
    f = L.etg_logits_i8

    def call(w=_p(), ws=64, sw=_p(), sws=1, vocab=100, hidden=64, r=_p(), dt=etg.F32, rs=64, batch=4, out=_p(),
             odt=etg.F32, os_=100, work=_p(), nbytes=1 << 40):
        return f(w, ws, sw, sws, vocab, hidden, r, dt, rs, batch, out, odt, os_, work, nbytes, None)
    assert call(batch=-1) == -3 and call(batch=65537) == -3 and call(vocab=-1) == -3 and call(hidden=0) == -3
    assert call(dt=etg.Q8_0) == -2 and "dtype" in _err(L)
    assert call(odt=7) == -2 and "output dtype" in _err(L)
    assert call(ws=63) == -3 and "w stride" in _err(L)
    assert call(rs=63) == -3 and "input stride" in _err(L)
    assert call(os_=99) == -3 and call(sws=0) == -3
    for name in ("w", "sw", "r", "out", "work"):
        assert call(**{name: None}) == -1, name
    assert call(r=_p(2)) == -4 and call(sw=_p(2)) == -4 and call(out=_p(2)) == -4 and call(work=_p(16)) == -4
    need = L.etg_logits_i8_workspace(4, 100, 64)
    assert need > L.etg_matmul_i8_workspace(4, 100, 64)
    assert call(nbytes=need - 1) == -6 and "workspace" in _err(L)
    assert call(batch=0, r=None, out=None, work=None) == 0 and call(vocab=0, w=None, out=None, work=None) == 0
    assert L.etg_logits_i8_workspace(65537, 1, 1) == -3


def _how(T=1.0, k=0, p=1.0, mp=0.0, dT=None, dk=None, dp=None, dmp=None, allowed=None, stride=0):
    return etg._Sampling(T, k, p, mp, dT, dk, dp, dmp, allowed, stride)


def test_sample_errors(L):
    f = L.etg_sample

    def call(x=_p(), dt=etg.F32, batch=4, vocab=100, stride=100, how=None, u=_p(), ids=_p(), probs=_p(), work=_p(),
             nbytes=1 << 40):
        h = how if how is not None else _how()
        return f(x, dt, batch, vocab, stride, ctypes.addressof(h), u, ids, probs, work, nbytes, None)
    assert call(dt=etg.Q8_0) == -2 and "dtype" in _err(L)
    assert call(batch=-1) == -3 and call(batch=65537) == -3
    assert call(vocab=0) == -3 and call(vocab=(1 << 20) + 1, stride=1 << 25) == -3 and "vocab" in _err(L)
    assert call(stride=99) == -3 and "stride" in _err(L)
    assert f(_p(), etg.F32, 4, 100, 100, None, _p(), _p(), _p(), _p(), 1 << 40, None) == -1
    for T in (-1.0, float("nan"), float("inf")):
        assert call(how=_how(T=T)) == -5 and "temperature" in _err(L)
    assert call(how=_how(k=-1)) == -5 and "top_k" in _err(L)
    for p in (0.0, -0.5, 1.5, float("nan")):
        assert call(how=_how(p=p)) == -5 and "top_p" in _err(L)
    for mp in (-0.1, 1.1, float("nan")):
        assert call(how=_how(mp=mp)) == -5 and "min_p" in _err(L)
    for name in ("x", "u", "ids", "probs"):
        assert call(**{name: None}) == -1, name
    assert call(x=_p(2)) == -4 and call(dt=etg.BF16, x=_p(1)) == -4
    for name in ("u", "ids", "probs"):
        assert call(**{name: _p(2)}) == -4, name
    assert call(how=_how(dT=FAKE + 2)) == -4 and call(how=_how(dk=FAKE + 1)) == -4
    assert call(how=_how(allowed=FAKE + 2)) == -4
    assert call(how=_how(allowed=FAKE, stride=3)) == -3 and "allowed" in _err(L)
    need = L.etg_sample_workspace(4, 100)
    assert need >= 0
    if need:
        assert call(work=None) == -1 and call(work=_p(16)) == -4
        assert call(nbytes=need - 1) == -6 and "workspace" in _err(L)
    assert call(batch=0, x=None, u=None, ids=None, probs=None) == 0
    assert L.etg_sample_workspace(-1, 5) == -3 and L.etg_sample_workspace(1, 0) == -3


def test_workspaces_depend_on_sizes_alone_and_cover_every_shape(L):
    for m in (0, 1, 8, 9, 16, 17, 64, 65, 256, 1024, 65536):
        for n in (0, 1, 33, 151936, 262144, 2 ** 31 - 1):
            for k in (1, 33, 896, 5376, 65536):
                b = L.etg_matmul_i8_workspace(m, n, k)
                assert b >= 0 and b == L.etg_matmul_i8_workspace(m, n, k)
    for batch in (0, 1, 64, 1024, 65536):
        for vocab in (1, 4096, 151936, 262144, 1 << 20):
            assert L.etg_sample_workspace(batch, vocab) >= 0


def test_python_refusals_on_host_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        etg.quantize_i8(x)
    with pytest.raises(ValueError):
        etg.quantize_i8(x.to(torch.float64))
    q = torch.zeros((4, 8), dtype=torch.int8)
    with pytest.raises(ValueError):
        etg.matmul_i8(q, torch.ones(4), q, torch.ones(4))
    with pytest.raises(ValueError):
        etg.matmul_i8(x, torch.ones(4), q, torch.ones(4))
    with pytest.raises(ValueError):
        etg.sample(x, torch.zeros(4))
    with pytest.raises(ValueError):
        etg.I8Table(q, torch.ones(4))


def test_rows_that_span_more_than_an_address_space(L):
    # (rows - 1) * stride * size past 2^57 bytes, up to 2^73: the kernels' 64-bit offsets would wrap
    M, far = 2 ** 31 - 1, 2 ** 40
    args = dict(x=_p(), dt=etg.F32, rows=M, cols=64, xs=64, q=_p(), qs=64, s=_p(), ss=1)
    for name, word in (("xs", "input stride"), ("qs", "code stride"), ("ss", "scale stride")):
        assert L.etg_quantize_i8(*{**args, name: far}.values(), None) == -3 and word in _err(L) and "2^57" in _err(L)
    # 2^16 rows 2^40 values apart are 2^56 bytes of codes, 2^57 of 16-bit values, 2^58 of f32 ones
    args = dict(a=_p(), as_=64, sa=_p(), sas=1, w=_p(), ws=64, sw=_p(), sws=1, m=4, n=M, k=64, out=_p(), dt=etg.F32,
                os_=M, work=_p(16), nbytes=0)
    for name, word in (("ws", "w stride"), ("sws", "w scale stride")):
        assert L.etg_matmul_i8(*{**args, name: far}.values(), None) == -3 and word in _err(L) and "2^57" in _err(L)
    args.update(m=65536, n=33001, os_=33001)
    for name, word in (("sas", "a scale stride"), ("os_", "output stride")):
        assert L.etg_matmul_i8(*{**args, name: far}.values(), None) == -3 and word in _err(L) and "2^57" in _err(L)
    # within it: past the strides' checks, to the workspace's alignment
    assert L.etg_matmul_i8(*{**args, "as_": far}.values(), None) == -4
    assert L.etg_matmul_i8(*{**args, "os_": far, "dt": etg.F16}.values(), None) == -4
    assert L.etg_logits_i8(_p(), far, _p(), 1, M, 64, _p(), etg.F32, 64, 4, _p(), etg.F32, M, _p(), 1 << 40, None) == -3
    assert "w stride" in _err(L) and "2^57" in _err(L)
    assert L.etg_logits_i8(_p(), 64, _p(), 1, 100, 64, _p(), etg.F32, far, 65536, _p(), etg.F32, 100, _p(), 1 << 50,
                           None) == -3
    assert "input stride" in _err(L) and "2^57" in _err(L)

    def sampled(how, dt=etg.F32, stride=100):
        return L.etg_sample(_p(), dt, 65536, 100, stride, ctypes.addressof(how), _p(), _p(), _p(), _p(16), 0, None)
    assert sampled(_how(), stride=far) == -3 and "logits stride" in _err(L) and "2^57" in _err(L)
    assert sampled(_how(), etg.BF16, far) == -4
    assert sampled(_how(allowed=FAKE, stride=far)) == -3 and "allowed stride" in _err(L) and "2^57" in _err(L)


@pytest.mark.parametrize("m,n,k", [(64, 33001, 256), (300, 33001, 1001), (17, 2 ** 20, 16)])
def test_matmul_workspace_refusals(L, m, n, k):
    # shapes of the kernels that read the a rows' image from the workspace
    need = L.etg_matmul_i8_workspace(m, n, k)
    assert need > 0

    def call(work=_p(), nbytes=need):
        return L.etg_matmul_i8(_p(), k, _p(), 1, _p(), k, _p(), 1, m, n, k, _p(), etg.F32, n, work, nbytes, None)
    assert call(work=None) == -1 and "workspace" in _err(L)
    assert call(work=_p(16)) == -4 and "256-byte aligned" in _err(L)
    assert call(nbytes=need - 1) == -6 and str(need) in _err(L)
    assert call(nbytes=0) == -6


@pytest.mark.parametrize("batch,vocab", [(1, 1), (4, 100), (64, 262144)])
def test_sample_workspace_refusals(L, batch, vocab):
    need = L.etg_sample_workspace(batch, vocab)
    assert need > 0
    how = _how()

    def call(work=_p(), nbytes=need):
        return L.etg_sample(_p(), etg.BF16, batch, vocab, vocab, ctypes.addressof(how), _p(), _p(), _p(), work, nbytes,
                            None)
    assert call(work=None) == -1 and "workspace" in _err(L)
    assert call(work=_p(16)) == -4 and "256-byte aligned" in _err(L)
    assert call(nbytes=need - 1) == -6 and str(need) in _err(L)
