"""The cross entropy's gradient of targets that are nearly certain: their entry of
g, p - 1, is far smaller than p is rounded by.

Logits are exact here: a row of the table is one column, a residual one column, so
that the target's logit is a and all others are 0: loss = log(1 + (V - 1) e^-a), which the
kernel keeps to 2^-13 of itself (test_loss), plus what exponentials below 2^-126
make.  Column 5 of dx is the target's entry alone: (p - 1) dloss.

Given the losses: expm1(-loss), good to that, 2^-22 and u^2 (two 16-bit terms) of
itself; f16 keeps 2^-40 of the largest |dloss| at least.  Without them: by the
definition expm1(z - lse) for the lse that is given; z - lse is one exact subtraction
here, rounded to 2^-24 of itself, expm1 good to 2^-22.
"""
import ctypes

import pytest
import torch

import embedding_lookup_tied_gb300 as lhs
from test_loss import CODE, FAKE, c_table, make, reference, check_grad, table_of

HALF = [torch.bfloat16, torch.float16]
V, H = 600, 64


def certain(t, dtype):
    """Losses from 2 down to 1e-8, a target that is one row for all."""
    w = torch.zeros((V, H), dtype=dtype, device="cuda")
    w[5, 5] = 1.0
    x = torch.zeros((t, H), dtype=dtype, device="cuda")
    x[:, 5] = (torch.arange(t, device="cuda") % 81) * 0.25 + 5.0
    y = torch.full((t,), 5, dtype=torch.int32, device="cuda")
    z = x[:, 5].double()
    loss = torch.log1p((V - 1) * torch.exp(-z))
    return w, x, y, z, loss


@pytest.mark.gpu
@pytest.mark.parametrize("temperature", [1.0, 2.0])
@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("t", [1, 81, 128, 129, 500])
def test_entries_keep_their_relative_accuracy(t, dtype, temperature):
    w, x, y, z, want = certain(t, dtype)
    x = (x.float() * temperature).to(dtype)
    tab = table_of(w)
    dl = torch.full((t,), 0.75, device="cuda")
    loss, lse, err = lhs.lhs_loss(tab, x, y, temperature=temperature)
    u = torch.finfo(dtype).eps / 2
    for given in (True, False):
        dx, dw = torch.empty((t, H), device="cuda"), torch.empty((V, H), device="cuda")
        lhs.lhs_loss_grad(tab, x, y, lse, dl, temperature=temperature, dx=dx, dtable=dw, err=err, loss=loss if given else None)
        entry = torch.expm1(-want if given else z - lse.double()) * (0.75 / temperature)
        tol = (u * u + 2.0 ** -22 + (2.0 ** -13 if given else 2.0 ** -22)) * entry.abs() + 0.75 / temperature * 2.0 ** -40
        d = (dx[:, 5].double() - entry).abs()
        assert bool((d <= tol).all()), (given, float((d / tol).max()))
        row = (entry * x[:, 5].double()).sum()
        tol = (tol * x[:, 5].double()).sum() + t * 2.0 ** -23 * row.abs()
        assert abs(float(dw[5, 5].double() - row)) <= float(tol), given
        assert bool((dx[:, :5] == 0).all()) and bool((dx[:, 6:] == 0).all())
    assert int(err.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("t", [60, 300])
def test_losses_are_used_only_where_positions_take_part(t):
    w, x, y, dl = make(t, 900, 72, torch.bfloat16, masked=0.4)
    y[0], y[1] = -100, 900
    r = reference(w, x, y, dl)
    tab = table_of(w)
    loss, lse, err = lhs.lhs_loss(tab, x, y)
    loss[~r["on"]] = float("nan")
    dx, dw, _ = lhs.lhs_loss_grad(tab, x, y, lse, dl, loss=loss, err=err)
    assert int(err.item()) == lhs.LHS_ERRBIT_BAD_TOKEN
    check_grad(dx, dw, r)
    k = int(r["on"].nonzero()[0])
    loss[k] = float("nan")
    dx, dw, err = lhs.lhs_loss_grad(tab, x, y, lse, dl, loss=loss)
    assert int(err.item()) & lhs.LHS_ERRBIT_NONFINITE
    assert bool(dx[k].isnan().any()) and bool(dw[int(y[k])].isnan().any())


def test_refusals():
    L, t = lhs.lib(), c_table()
    need = ctypes.c_size_t()
    assert L.lhs_loss_grad_workspace(ctypes.byref(t), 5, ctypes.byref(need)) == 0
    G = 1 << 30

    def call(x=1 * G, y=2 * G, loss=3 * G, lse=4 * G, dl=5 * G, dx=6 * G, dw=7 * G, ws=8 * G, err=9 * G, n=5, acc=0):
        return L.lhs_loss_grad_of(ctypes.byref(t), x, lhs.LHS_BF16, 64, n, y, -100, 1.0, loss, lse, dl, dx, lhs.LHS_BF16, 64,
                                  dw, lhs.LHS_BF16, acc, ws, need.value, err, None)
    for bad in (dict(loss=3 * G + 2), dict(lse=None), dict(dl=None), dict(acc=3), dict(dw=3 * G), dict(dx=3 * G), dict(ws=3 * G),
                dict(err=3 * G + 8), dict(loss=8 * G + 256)):
        assert call(**bad) == lhs.LHS_ERR_INVALID_ARG, bad
    assert call(n=0, acc=1, x=None, y=None, loss=None, lse=None, dl=None, ws=None, err=None) == lhs.LHS_OK
    assert t.data == FAKE and CODE[torch.bfloat16] == t.dtype
