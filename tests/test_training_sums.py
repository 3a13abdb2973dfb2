"""The oracle of the cross entropy gradients' sums, on the CPU: exact sums pass, sums that lost some rows,
or took them twice, do not."""
import pytest
import torch

from tests import training_sums as ts


@pytest.mark.parametrize("case", ts.CASES, ids=str)
def test_lost_rows_are_outside(case):
    dtype, n, V, d = ts.TYPES[case[0]], *case[1:]
    E, x, labels, h = ts.make(n, V, d, dtype)
    half = d // 2
    wx, wE = ts.want(E, x, h)
    tx, tE = ts.bound(wx, n, V, d, dtype), ts.bound(wE, n, n, d, dtype) if ts.exact_d(n, V, d, dtype) else None
    assert ((wx.to(dtype).double() - wx).abs() <= tx).all()
    # 16 bits: a stage of 64 table rows lost or taken twice; f32 D: a slice of an eighth (one pass: 1 / 512) of them
    lost = 64 if ts.exact_d(n, V, d, dtype) else V // 512 if ts.one_pass(n, V, d, dtype) else V // 8
    for v0 in (0, V // 2 // 64 * 64, V - lost):
        part = E[v0:v0 + lost, 1:half].double().sum(0) * (h.double() / V)[:, None]
        for sign in (-1, 1):
            got = (wx + sign * part).to(dtype).double()
            assert ((got - wx).abs() > tx).any(), (v0, sign)
    if tE is not None:  # one residual row lost, where there are few enough for 8 bits
        for b in (0, n // 2, n - 1) if n <= 128 else ():
            got = (wE - (h.double() / V)[b] * x[b, half:].double()).to(dtype).double()
            assert ((got - wE).abs() > tE).any(), b
