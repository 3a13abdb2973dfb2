"""Refusals of the tied table's training operators, on the host: nothing is launched."""
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


def _table(L, dtype=etg.BF16, V=1000, d=64):
    h = ctypes.c_void_p()
    assert L.etg_table_create(_p(), dtype, V, d, ctypes.byref(h)) == 0
    return h


def test_cross_entropy_errors(L):
    t, q8 = _table(L), _table(L, etg.Q8_0)

    def call(t=t, x=_p(), xs=64, n=4, y=_p(), loss=_p(), lse=_p(), work=_p(), nbytes=1 << 40):
        return L.etg_cross_entropy(t, x, xs, n, y, loss, lse, work, nbytes, None)
    assert call(t=None) == -1 and "table" in _err(L)
    assert call(t=q8) == -2 and "Q8_0" in _err(L)
    assert call(n=-1) == -3 and call(n=65537) == -3 and "batch" in _err(L)
    assert call(xs=63) == -3 and "residual stride" in _err(L)
    assert call(xs=2 ** 40 + 1) == -3
    for name in ("x", "y", "loss", "lse"):
        assert call(**{name: None}) == -1, name
    for name in ("y", "loss", "lse"):
        assert call(**{name: _p(2)}) == -4, name
    assert call(x=_p(1)) == -4 and "residual" in _err(L)
    need = L.etg_cross_entropy_workspace(t, 4)
    assert need > 0
    assert call(work=None) == -1 and call(work=_p(16)) == -4
    assert call(nbytes=need - 1) == -6 and str(need) in _err(L)
    assert call(n=0, x=None, y=None, loss=None, lse=None, work=None, nbytes=0) == 0
    assert L.etg_cross_entropy_workspace(t, 0) == 0
    assert L.etg_cross_entropy_workspace(t, 65537) == -3 and L.etg_cross_entropy_workspace(q8, 4) == -2
    assert L.etg_cross_entropy_workspace(None, 4) == -1


def test_cross_entropy_grad_errors(L):
    t, q8, f32 = _table(L), _table(L, etg.Q8_0), _table(L, etg.F32)

    def call(t=t, x=_p(), xs=64, n=4, y=_p(), lse=_p(), g=1.0, dg=None, dh=None, dx=_p(), dxs=64, dE=_p(), add=0,
             work=_p(), nbytes=1 << 40):
        return L.etg_cross_entropy_grad(t, x, xs, n, y, lse, g, dg, dh, dx, dxs, dE, add, work, nbytes, None)
    assert call(t=None) == -1 and call(t=q8) == -2
    assert call(n=-1) == -3 and call(n=65537) == -3
    assert call(xs=63) == -3 and call(dxs=63) == -3 and "residual gradient stride" in _err(L)
    for name in ("x", "y", "lse"):
        assert call(**{name: None}) == -1, name
    for name in ("y", "lse", "dg", "dh"):
        assert call(**{name: _p(2)}) == -4, name
    assert call(x=_p(1)) == -4 and call(dx=_p(1)) == -4 and call(t=f32, dx=_p(2)) == -4
    assert call(dE=_p(8)) == -4 and "table gradient" in _err(L)
    need = L.etg_cross_entropy_grad_workspace(t, 4)
    assert need > 0
    assert call(work=None) == -1 and call(work=_p(16)) == -4
    assert call(nbytes=need - 1) == -6 and str(need) in _err(L)
    assert call(dx=None, dE=None, work=None) == 0          # nothing is wanted
    assert call(dx=None, dxs=0, work=None) == -1           # its stride is not looked at
    assert call(n=0, x=None, y=None, lse=None, dx=None, dE=None, work=None, nbytes=0) == 0
    assert call(n=0, x=None, y=None, lse=None, add=1, work=None, nbytes=0) == 0  # leaves the table's as it is
    assert L.etg_cross_entropy_grad_workspace(t, 0) == 0
    assert L.etg_cross_entropy_grad_workspace(t, -1) == -3 and L.etg_cross_entropy_grad_workspace(q8, 1) == -2


def test_embed_gather_grad_errors(L):
    t, q8 = _table(L), _table(L, etg.Q8_0)

    def call(t=t, ids=_p(), n=4, g=_p(), gt=etg.F32, gs=64, out=_p(), ot=etg.BF16, add=0, work=_p(), nbytes=1 << 40):
        return L.etg_embed_gather_grad(t, ids, n, g, gt, gs, 1.0, out, ot, add, work, nbytes, None)
    assert call(t=None) == -1 and call(t=q8) == -2
    assert call(n=-1) == -3 and call(n=2 ** 24 + 1) == -3 and "seq_len" in _err(L)
    assert call(gt=etg.Q8_0) == -2 and call(gt=9) == -2
    assert call(ot=etg.F16) == -2 and "output dtype" in _err(L)
    assert call(gs=63) == -3 and "gradient stride" in _err(L)
    for name in ("ids", "g", "out"):
        assert call(**{name: None}) == -1, name
    assert call(ids=_p(2)) == -4 and call(g=_p(2)) == -4 and call(gt=etg.F16, g=_p(1)) == -4
    assert call(out=_p(8)) == -4
    need = L.etg_embed_gather_grad_workspace(t, 4)
    assert need > 0
    assert call(work=None) == -1 and call(work=_p(16)) == -4
    assert call(nbytes=need - 1) == -6 and str(need) in _err(L)
    assert call(n=0, ids=None, g=None, add=1, work=None, nbytes=0) == 0
    assert L.etg_embed_gather_grad_workspace(t, 0) == 0
    assert L.etg_embed_gather_grad_workspace(t, 2 ** 24 + 1) == -3 and L.etg_embed_gather_grad_workspace(q8, 1) == -2


def test_rows_that_span_more_than_an_address_space(L):
    t = _table(L, etg.F32)
    far = 2 ** 40
    assert L.etg_cross_entropy(t, _p(), far, 65536, _p(), _p(), _p(), _p(), 1 << 50, None) == -3 and "2^57" in _err(L)
    assert L.etg_cross_entropy_grad(t, _p(), 64, 65536, _p(), _p(), 1.0, None, None, _p(), far, None, 0, _p(), 1 << 50,
                                    None) == -3 and "2^57" in _err(L)
    assert L.etg_embed_gather_grad(t, _p(), 2 ** 24, _p(), etg.F32, far, 1.0, _p(), etg.F32, 0, _p(), 1 << 50,
                                   None) == -3 and "2^57" in _err(L)


def test_workspaces_stay_bounded(L):
    # beyond the residual rows' own size: statistics, D and the partial sums of a few hundred MiB
    for dtype, unit in ((etg.F32, 4), (etg.BF16, 2), (etg.F16, 2)):
        for V in (1, 257, 4096, 262144, 2 ** 31 - 1):
            for d in (8, 896, 5376, 65536):
                t = _table(L, dtype, V, d)
                for n in (1, 2, 64, 65, 1000, 4096, 65536):
                    rows = n * d * unit
                    f = L.etg_cross_entropy_workspace(t, n)
                    assert 0 < f <= rows + (257 << 20) + 4096
                    b = L.etg_cross_entropy_grad_workspace(t, n)
                    assert 0 < b <= rows + (257 << 20) + 4096 + 1024 * max(n, 256) * 256 * 4 + n * d * 4
                    r = L.etg_embed_gather_grad_workspace(t, n)
                    assert 0 < r <= (260 << 20) + 64 * d + 16 * n + 4 * 512 * (n // 4096 + 1) * 4
                    assert f == L.etg_cross_entropy_workspace(t, n)
                L.etg_table_destroy(t)
        t = _table(L, dtype, 2 ** 31 - 1, 65536)
        assert 0 < L.etg_embed_gather_grad_workspace(t, 2 ** 24) < (1 << 30)


def test_python_refusals_on_host_tensors():
    with pytest.raises(ValueError):
        etg.Table(torch.zeros(4, 8), etg.F32, 4, 8)
    t = etg.Table.__new__(etg.Table)  # a table's arguments without a device
    t.dtype, t.vocab, t.hidden, t.device = etg.BF16, 4, 8, torch.device("cpu")
    x, y, f = torch.zeros((3, 8), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32), torch.zeros(3)
    for bad in (x.float(), x.half()):
        with pytest.raises(ValueError, match="table's type"):
            t.cross_entropy(bad, y)
    with pytest.raises(ValueError):
        t.cross_entropy(x, y)  # not on a GPU
    with pytest.raises(ValueError):
        t.cross_entropy_grad(x, y, f)
    with pytest.raises(ValueError, match="int32"):
        t.embed_gather_grad(torch.zeros((3, 8)), y.long())
    with pytest.raises(ValueError, match="grad must be"):
        t.embed_gather_grad(torch.zeros((3, 8), dtype=torch.float64), y)
    with pytest.raises(ValueError):
        t.embed_gather_grad(torch.zeros((3, 8)), y)
    with pytest.raises(ValueError, match="accumulate"):
        t._table_grad(None, (torch.bfloat16,), torch.bfloat16, True)
    with pytest.raises(ValueError, match="contiguous"):
        t._table_grad(torch.zeros((4, 8)), (torch.bfloat16,), torch.bfloat16, False)
    t.dtype = etg.Q8_0
    for call in (lambda: t.cross_entropy(x, y), lambda: t.cross_entropy_grad(x, y, f),
                 lambda: t.embed_gather_grad(torch.zeros((3, 8)), y)):
        with pytest.raises(ValueError, match="Q8_0"):
            call()
