"""Gradients that are sums of very many terms of one sign, over positions (dtable)
and over the vocabulary (dx).

Bounds, of the sum A of the terms' magnitudes, which all have one sign.  The tensor cores
cut each of a step's 17 addends at 2^-25 of the largest (test_loss_long_rows):
2,048 terms are 128 steps, 128 17 2^-26 of their sum.  Such parts are added in f32,
n / 2048 additions of 2^-24 of half of A on average.  The targets' rows are f32 sums
of runs of at most 128 positions, which 16 warps add up: (64 + n / 4096 + 16) 2^-24.
One sum would be short by n / 512 times 44 2^-24 (f16) or 3.5 2^-24 (bf16) of A: 2.7e-3
and 2.1e-4 for 2^19 terms, where the bounds are 4e-5.
"""
import pytest
import torch

import embedding_lookup_tied_gb300 as lhs
from test_loss import table_of

pytestmark = pytest.mark.gpu
HALF = [torch.bfloat16, torch.float16]


def parts(n):
    return 128 * 17 * 2.0 ** -26 + (n / 2048 + 1) / 2 * 2.0 ** -24


@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("t", [5000, 1 << 19])
def test_table_gradient_of_many_positions(t, dtype):
    # two words, no logits: p = 1/2 exactly (lse is given), every position has the first word's target
    v, h = 2, 40
    g = torch.Generator().manual_seed(t)
    w = torch.zeros((v, h), dtype=dtype, device="cuda")
    x = (torch.rand((t, h), generator=g) * 0.5 + 0.5).to(dtype).cuda()
    y = torch.zeros(t, dtype=torch.int32, device="cuda")
    lse = torch.full((t,), 0.6931471805599453, device="cuda")  # exp(-lse) is 1/2 to 2^-24 of itself
    for out in (torch.float32, dtype):
        dw = torch.empty((v, h), dtype=out, device="cuda")
        dl = torch.full((t,), 2.0 ** -12 if out == torch.float16 else 1.0, device="cuda")  # f16 ends at 65,504
        _, _, err = lhs.lhs_loss_grad(table_of(w), x, y, lse, dl, want_dx=False, dtable=dw)
        want = x.double().sum(0) * (0.5 * float(dl[0]))
        own = 2.0 ** -20 + torch.finfo(out).eps / 2 * 1.01 * (out != torch.float32)
        assert int(err.item()) == 0
        off = ((dw[1].double() - want).abs() / want).max()
        assert float(off) <= parts(t) + own, float(off)
        off = ((dw[0].double() + want).abs() / want).max()
        assert float(off) <= (80 + t / 4096) * 2.0 ** -24 + parts(t) * 2.0 ** -20 + own, float(off)


@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("t,v", [(1, 500000), (200, 300000), (3000, 20001)])
def test_residuals_gradient_of_many_words(t, v, dtype):
    # no residuals, so that every word has p = 1 / v; the terms are p times rows of one sign.  Above 128
    # positions p is rounded to 16 bits, the same for all words: its rounding u is one of the sum
    h = 24
    g = torch.Generator().manual_seed(v)
    w = (torch.rand((v, h), generator=g) * 0.5 + 0.5).to(dtype).cuda()
    x = torch.zeros((t, h), dtype=dtype, device="cuda")
    y = torch.arange(t, dtype=torch.int32, device="cuda") % v
    tab = table_of(w)
    _, lse, err = lhs.lhs_loss(tab, x, y)
    dx = torch.empty((t, h), device="cuda")
    lhs.lhs_loss_grad(tab, x, y, lse, torch.ones(t, device="cuda"), dx=dx, want_dtable=False, err=err)
    p = torch.exp(-lse.double())[:, None]
    want = p * w.double().sum(0) - w[y.long()].double()
    u = torch.finfo(dtype).eps / 2
    tol = (parts(v) + 2.0 ** -19 + (u * u if t <= 128 else u)) * (p * w.double().sum(0)) + 2.0 ** -20
    d = (dx.double() - want).abs()
    assert bool((d <= tol).all()), float((d / tol).max())
    assert int(err.item()) == 0
