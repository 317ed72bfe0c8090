"""The cross entropy's gradient where targets repeat, as words of a text do: a
row of the table's gradient is then a sum over many positions, whose terms
have different signs, and an element of it may be far below its terms.

Bounds per element.  The target's entry of g, (p - 1) dloss, is not rounded to 16
bits: p is off by 2 (E + dz) of itself (test_loss), the entry by 2^-22 of itself
besides.  The other entries are rounded once, u = eps / 2 of themselves (f16:
2^-39 of the largest |dloss| at least, as test_loss has it).  The rest as there: sums
in f32, and the result's own rounding.  (One rounding of the target's entry, u of
itself, leaves these bounds by far: 2^-9 of 30 terms against 2^-13.)
"""
import pytest
import torch

import embedding_lookup_tied_gb300 as lhs
from test_loss import E, make, reference, rounding, table_of, within

HALF = [torch.bfloat16, torch.float16]


def frequent(t, v, seed, masked=0.0):
    """Targets whose rank r has probability proportional to r^-1.1."""
    g = torch.Generator().manual_seed(seed)
    c = torch.cumsum(torch.arange(1, v + 1, dtype=torch.float64) ** -1.1, 0)
    r = torch.searchsorted(c, torch.rand(t, generator=g, dtype=torch.float64) * c[-1]).clamp(max=v - 1)
    y = torch.randperm(v, generator=g)[r].to(torch.int32)
    y[torch.rand(t, generator=g) < masked] = -100
    return y.cuda()


def bounds(w, x, y, dl):
    """(dx, dtable) by the formula, each with how far it may be off before its rounding; and the positions."""
    r = reference(w, x, y, dl)
    on = r["on"]
    W, X, d = w.double(), x[on].double(), dl[on].double()[:, None]
    at = y[on].long()[:, None]
    p = torch.exp(X @ W.T - r["lse"][:, None])
    u = torch.finfo(w.dtype).eps / 2
    tiny = float(d.abs().max()) * 2.0 ** -39 if w.dtype == torch.float16 and len(d) else 0.0
    dg = (u + 2 * E) * p * d.abs() + tiny
    pt = p.gather(1, at)
    dg.scatter_(1, at, 2 * E * pt * d.abs() + 2.0 ** -22 * (1 - pt) * d.abs() + tiny)
    mag = p * d.abs()
    mag.scatter_(1, at, (1 - pt) * d.abs())
    dx_tol = dg @ W.abs() + w.shape[0] * 2.0 ** -23 * (mag @ W.abs())
    dw_tol = dg.T @ X.abs() + (len(X) + 2) * 2.0 ** -23 * (mag.T @ X.abs())
    return r, dx_tol, dw_tol


def check(w, x, y, dl, out):
    tab = table_of(w)
    r, dx_tol, dw_tol = bounds(w, x, y, dl)
    on = r["on"]
    _, lse, err = lhs.lhs_loss(tab, x, y)
    dx = torch.empty(x.shape, dtype=out, device="cuda")
    dw = torch.full(w.shape, float("nan"), dtype=out, device="cuda")
    lhs.lhs_loss_grad(tab, x, y, lse, dl, dx=dx, dtable=dw, err=err)
    assert int(err.item()) == 0
    within(dx[on], r["dx"], dx_tol + rounding(r["dx"], out) * 1.01)
    assert bool((dx[~on] == 0).all())
    within(dw, r["dw"], dw_tol + rounding(r["dw"], out) * 1.01)
    return r, dw


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["table", "f32"])
@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("t,v,h", [(256, 100003, 128), (1024, 100003, 64), (1000, 130000, 72), (300, 9001, 1001), (129, 500, 33)])
def test_rows_of_frequent_targets(t, v, h, dtype, out):
    w, x, _, dl = make(t, v, h, dtype)
    check(w, x, frequent(t, v, t + h, 0.1), dl, dtype if out == "table" else torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF, ids=str)
def test_error_in_norm_is_that_of_one_rounding(dtype):
    """Probabilities of 16 bits in g are a term of their own, which the targets' rows do not feel: in norm over
    the table's gradient, sqrt(1 + s^2) of the result's rounding, where s is the norm of the other entries'
    part against the whole, at most; and 2^-12 for the f32 steps."""
    t, v, h = 512, 50000, 256
    w, x, _, _ = make(t, v, h, dtype, masked=0.0)
    y = frequent(t, v, 5)
    dl = torch.rand(t, generator=torch.Generator().manual_seed(1)).cuda() + 0.5
    r, dw = check(w, x, y, dl, dtype)
    once = float((r["dw"].to(dtype).double() - r["dw"]).norm() / r["dw"].norm())
    p = torch.exp(x.double() @ w.double().T - r["lse"][:, None])
    p.scatter_(1, y.long()[:, None], 0.0)
    s = float(((p * dl.double()[:, None]).T @ x.double()).norm() / r["dw"].norm())
    got = float((dw.double() - r["dw"]).norm() / r["dw"].norm())
    assert got <= once * (1 + s * s) ** 0.5 * 1.02 + 2.0 ** -12, (got, once, s)


@pytest.mark.gpu
@pytest.mark.parametrize("t", [129, 3000, 9000])
def test_one_target_everywhere_and_each_once(t):
    # a row of all positions (runs that cross, joined), a row each, rows that lie by id and by place
    for v, h in ((40, 72), (20000, 24), (t, 8)):
        w, x, _, dl = make(t, v, h, torch.bfloat16)
        check(w, x, torch.full((t,), v - 1, dtype=torch.int32, device="cuda"), dl, torch.float32)
        check(w, x, (torch.randperm(t, generator=torch.Generator().manual_seed(t)) % v).to(torch.int32).cuda(), dl, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("h", [64, 100])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=str)
def test_added_to_what_the_gradient_held(h, out):
    t, v = 400, 5000
    w, x, _, dl = make(t, v, h, torch.bfloat16)
    y = frequent(t, v, 3, 0.2)
    r, _, dw_tol = bounds(w, x, y, dl)
    tab = table_of(w)
    _, lse, err = lhs.lhs_loss(tab, x, y)
    base = torch.randn((v, h), generator=torch.Generator().manual_seed(2)).to(out).cuda()
    got = base.clone()
    lhs.lhs_loss_grad(tab, x, y, lse, dl, want_dx=False, dtable=got, accumulate=True, err=err)
    ref = r["dw"] + base.double()
    within(got, ref, dw_tol + 2.0 ** -23 * r["dw"].abs() + rounding(ref, out) * 1.01)
    assert int(err.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("t", [90, 300])
def test_upstream_gradients_far_apart(t):
    """bf16: every row of dx is as accurate as if it stood alone, whatever the others' dloss.  f16: down to
    2^-40 of the largest |dloss| (test_loss's 2^-39, doubled for what is cut off), in whose units a row is
    off; the targets' entries of more than 128 positions are not."""
    v, h = 700, 64
    step = 2.0 ** -(torch.arange(t) % 46).float().cuda()
    for dtype in HALF:
        w, x, y, _ = make(t, v, h, dtype, masked=0.1)
        r, dx_tol, dw_tol = bounds(w, x, y, step)
        on = r["on"]
        tab = table_of(w)
        _, lse, err = lhs.lhs_loss(tab, x, y)
        dx, dw = torch.empty((t, h), device="cuda"), torch.empty((v, h), device="cuda")
        lhs.lhs_loss_grad(tab, x, y, lse, step, dx=dx, dtable=dw, err=err)
        within(dx[on], r["dx"], dx_tol)
        within(dw, r["dw"], dw_tol)
        assert int(err.item()) == 0
        if t > 128:  # what is left of a row that f16's g has lost: the target's part
            far = on & (step < 2.0 ** -41)
            alone = (torch.exp(-r["loss"]) - 1)[:, None] * step[on].double()[:, None] * w[y[on].long()].double()
            here = (step[on] < 2.0 ** -41)
            assert dtype == torch.bfloat16 or bool((dx[far].double() - alone[here]).abs().max() <= 2.0 ** -12 * alone[here].abs().max())
            assert bool((dx[far] != 0).any())
