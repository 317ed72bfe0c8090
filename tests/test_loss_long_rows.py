"""Logits that are long sums of one sign: tensor cores cut an f32 sum instead of
rounding it, always towards zero, so that one sum over all of hidden falls
short by what it was cut; the loss and its gradient sum 512 of hidden at a time.

Bound of such a logit of magnitude A, all of whose terms are positive.  A step adds 16
products to the sum; the 17 addends are lined up with the largest, and what lies below
2^-25 of it is cut off each (two bits more than an f32 keeps, which is known of these tensor
cores from published measurements; the sums of 512 below agree with it: f16 products of 22
bits lose half of that each, 44 2^-24 of the sum, bf16 products of 16 bits mostly end before it,
3.5 2^-24).  So a step cuts at most 17 2^-25 of the running sum, which is half of the 512's on
average: 32 17 2^-26 of each 512's part, and so of A.  The parts are then added, rounded:
H / 512 additions of 2^-24 of half of A on average.  One long sum would be short by H / 512 times
44 (or 3.5) 2^-24 of A.
"""
import pytest
import torch

import embedding_lookup_tied_gb300 as lhs
from test_loss import make, table_of, within

pytestmark = pytest.mark.gpu
HALF = [torch.bfloat16, torch.float16]


def dz(h, a):
    return a * (32 * 17 * 2.0 ** -26 + (h / 512 + 1) / 2 * 2.0 ** -24)


def positive(shape, g, size):
    return (torch.rand(shape, generator=g) * 0.5 + 0.5) * size


@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("h", [5376, 20000, 65536])
def test_loss_of_long_rows(h, dtype):
    """The target's logit is about 30, the others' 22 exactly (one product each), V = e^8: the loss is
    about ln 2, and its error (1 - p) of the logit's.  lse besides: an exponential is good to 2^-21, its
    argument to 2^-24 of up to 2^6, and 128 + V / 128 additions of 2^-24 of the sum."""
    v, t = 2980, 40
    g = torch.Generator().manual_seed(h)
    w = torch.zeros((v, h))
    w[:, 0] = 2.0
    x = torch.zeros((t, h))
    x[:, 0] = 11.0
    y = torch.randint(0, v, (t,), generator=g, dtype=torch.int32)
    y[:] = torch.unique(torch.cat([y, torch.arange(t, dtype=torch.int32)]))[:t]
    w[y.long()] = 0.0
    for i in range(t):  # a row of its own for each position, over columns that no other row has
        w[y[i].long(), 1:] = positive((h - 1,), g, 2.0 ** -4)
    x[:, 1:] = positive((t, h - 1), g, 30.0 / (0.75 ** 2 * (h - 1) * 2.0 ** -4))
    w, x, y = w.to(dtype).cuda(), x.to(dtype).cuda(), y.cuda()
    # positions see one another's rows as well: one position at a time
    for i in range(0, t, 13):
        only = w.clone()
        only[y.long()] = 0.0
        only[y.long(), 0] = 2.0
        only[y[i].long()] = w[y[i].long()]
        z = x[i].double() @ only.double().T
        a = float(z.max())
        want = float(torch.logsumexp(z, 0) - z[y[i].long()])
        p = float(torch.exp(z[y[i].long()] - torch.logsumexp(z, 0)))
        loss, lse, err = lhs.lhs_loss(table_of(only), x[i:i + 1], y[i:i + 1])
        tol = (1 - p) * dz(h, a) + 2.0 ** -21 + 2.0 ** -18 + (128 + v / 128) * 2.0 ** -24 * (1 - p) + 2.0 ** -23 * (a + 1)
        assert abs(float(loss) - want) <= tol, (float(loss) - want, tol)
        assert int(err.item()) == 0


@pytest.mark.parametrize("temperature", [1.0, 2.0])
@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("h", [5376, 20000, 65536])
def test_probabilities_sum_to_one(h, dtype, temperature):
    """A column of ones in the table that no residual has: its dx is (sum of p - 1) dloss.

    By the definition: sum of exp(z - lse) - 1 for the lse that is given; each p is off by dz of itself,
    an exponential's 2^-21 and its argument's 2^-24 of up to 2^5; g by u^2 of its magnitudes, which sum to
    2 at most (few positions); the sum over V by 17 / 16 2^-25 for each of it.

    By itself: the logits are the very ones that lse was summed from, so dz takes no part.  lse is good
    to 2^-24 of up to 2^6 in an exponential's argument, 2^-21 in its value, 64 2^-24 in their sum and
    2^-24 of up to 2^6 in its rounding; the rest as above.  (Logits of one long sum in g: 6e-5 at the least.)"""
    v, t = 600, 20
    g = torch.Generator().manual_seed(h)
    w, x = positive((v, h), g, 2.0 ** -4), positive((t, h), g, temperature * 30.0 / (0.75 ** 2 * (h - 1) * 2.0 ** -4))
    w[:, 7], x[:, 7] = 1.0, 0.0
    y = torch.randint(0, v, (t,), generator=g, dtype=torch.int32).cuda()
    w, x = w.to(dtype).cuda(), x.to(dtype).cuda()
    tab = table_of(w)
    _, lse, err = lhs.lhs_loss(tab, x, y, temperature=temperature)
    dx = torch.empty((t, h), device="cuda")
    lhs.lhs_loss_grad(tab, x, y, lse, torch.ones(t, device="cuda"), temperature=temperature, dx=dx, want_dtable=False, err=err)
    z = x.double() @ w.double().T / temperature
    want = (torch.exp(z - lse.double()[:, None]).sum(1) - 1) / temperature
    u = torch.finfo(dtype).eps / 2
    own = 2.0 ** -21 + 2.0 ** -19 + 2 * u * u + v * 17 / 16 * 2.0 ** -25
    tol = (dz(h, float(z.max())) + own) / temperature
    off = float((dx[:, 7].double() - want).abs().max())
    assert off <= tol, (off, tol)
    off, tol = float(dx[:, 7].abs().max()), (own + 3 * 2.0 ** -18 + 2.0 ** -21) / temperature
    assert off <= tol, (off, tol)
    assert int(err.item()) == 0


@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("t,v,h", [(100, 3000, 5376), (300, 2000, 5376), (260, 9000, 2000), (150, 700, 1033)])
def test_random_long_rows(t, v, h, dtype):
    """Loss and gradients of values of both signs, with the logits' bound above (A the sum of magnitudes, for
    the running sum stays below it), and the rest as in test_loss_targets."""
    w, x, y, dl = make(t, v, h, dtype, exact=False)
    W, X = w.double(), x.double()
    z = X @ W.T
    d = dz(h, float((X.abs() @ W.abs().T).max()))
    on = y >= 0
    n = torch.logsumexp(z, 1, keepdim=True)
    at = y.clamp(min=0).long()[:, None]
    want = (n - z.gather(1, at))[:, 0]
    tab = table_of(w)
    loss, lse, err = lhs.lhs_loss(tab, x, y)
    tol = 2 * d + 2.0 ** -18 + (128 + v / 128) * 2.0 ** -24 + 2.0 ** -22 * z.abs().amax(1)
    assert bool(((loss.double() - want).abs() <= tol)[on].all())
    dx, dw = torch.empty((t, h), device="cuda"), torch.empty((v, h), device="cuda")
    lhs.lhs_loss_grad(tab, x, y, lse, dl, dx=dx, dtable=dw, err=err)
    dd = dl.double()[:, None] * on[:, None]
    p = torch.exp(z - n)
    g = (p - torch.zeros_like(p).scatter_(1, at, 1.0)) * dd
    u = torch.finfo(dtype).eps / 2
    dp = 2 * d + 2.0 ** -17 + (128 + v / 128) * 2.0 ** -24
    few = int(on.sum()) <= 128
    dg = ((u * u if few else u) + dp) * p * dd.abs() + float(dl.abs().max()) * 2.0 ** -39
    pt = p.gather(1, at)
    dg.scatter_(1, at, ((dp + u * u) * pt + (2.0 ** -22 + (u * u if few else 0.0)) * (1 - pt)) * dd.abs() + float(dl.abs().max()) * 2.0 ** -39)
    within(dx, g @ W, dg @ W.abs() + v * 2.0 ** -23 * (g.abs() @ W.abs()))
    within(dw, g.T @ X, dg.T @ X.abs() + (t + 2) * 2.0 ** -23 * (g.abs().T @ X.abs()))
    assert int(err.item()) == 0


@pytest.mark.parametrize("temperature", [1.0, 0.5])
@pytest.mark.parametrize("top", [8.0, 250.0, 1000.0])
@pytest.mark.parametrize("dtype", HALF, ids=str)
def test_loss_of_large_logits(dtype, top, temperature):
    """Logits top - 0, 0.5, .. 3.5, exact in f32: the loss depends on their differences alone, and is as good
    where they are far from 0.  An exponential is good to 2^-21, its argument (a difference, scaled) to
    2^-23 of up to 7 log2(e) in its value, their sum to 48 2^-24 (128 in four, blocks, tiles and parts), the
    logarithm to 2^-22 of itself.  (Exponentials of z and of the maximum scaled apart: 2^-24 of
    1,443, 6e-5, at 1,000.)"""
    v, t, h = 3001, 9, 72
    w = torch.zeros((v, h), dtype=dtype, device="cuda")
    w[:, 0], w[:, 1] = 1.0, -(torch.arange(v, device="cuda") % 8 * 0.25)
    x = torch.zeros((t, h), dtype=dtype, device="cuda")
    x[:, 0], x[:, 1] = top, 2.0
    y = torch.arange(t, dtype=torch.int32, device="cuda") + 5
    loss, lse, err = lhs.lhs_loss(table_of(w), x, y, temperature=temperature)
    z = x.double() @ w.double().T / temperature
    want = torch.logsumexp(z - z[0, 0], 1) - (z.gather(1, y.long()[:, None])[:, 0] - z[0, 0])
    tol = 2.0 ** -21 + 7 * 1.45 / temperature * 2.0 ** -23 + 48 * 2.0 ** -24 + 2.0 ** -22 * 16
    off = float((loss.double() - want).abs().max())
    assert off <= tol, (off, tol)
    assert float((lse.double() - torch.logsumexp(z, 1)).abs().max()) <= tol + 2.0 ** -23 * (top / temperature + 8)
    assert int(err.item()) == 0
