"""Cross entropy over the tied table and its gradient, against the formulas in
64 bits.

Tolerances.  Where residuals and table hold small multiples of powers of two
every sum of products is exact in f32, so a logit is exact.  Else a logit is off
by at most H additions of a step 2^-23 each (a tensor core may cut instead of
round): H 2^-23 sum|x w|, called dz.  An exponential is good to 2^-21 and its
argument to 2^-23 of up to 2^7; a sum over the vocabulary in tiles of 256 has at
most 256 + V/256 + 5 additions of 2^-24 each: together below 2^-14 for V < 2^17,
an absolute error of lse, called E = 2^-14.  loss: twice E + dz, and its rounding.

Gradient.  p is off by E + dz of itself (twice: lse and logit).  g is then
rounded to the table's type: u = eps / 2 of itself, or half of the last subnormal
of f16 under the largest |g| scaled to 2^14 or more: 2^-39 of the largest.  The
sums over n terms in f32: n 2^-23 of the sum of magnitudes.  The result's own
rounding: its type's eps / 2 (f16 subnormals: 2^-25).
"""
import ctypes
import math

import pytest
import torch

import embedding_lookup_tied_gb300 as lhs

FAKE = 0x10000
E = 2.0 ** -14
CODE = {torch.float16: lhs.LHS_F16, torch.bfloat16: lhs.LHS_BF16}
HALF = [torch.bfloat16, torch.float16]


# ---------------------------------------------------------------------------
# refusals (host)
# ---------------------------------------------------------------------------
def c_table(dtype=lhs.LHS_BF16, vocab=1000, hidden=64):
    t = lhs.lhs_table()
    assert lhs.lib().lhs_table_init(ctypes.byref(t), FAKE, vocab, hidden, dtype) == 0
    return t


def test_loss_refuses():
    L, t = lhs.lib(), c_table()
    big = 1 << 40

    def call(t=t, x=FAKE, dt=lhs.LHS_BF16, stride=64, n=5, y=FAKE, temp=1.0, loss=FAKE, lse=FAKE, ws=FAKE, wb=big,
             err=FAKE):
        return L.lhs_loss(ctypes.byref(t), x, dt, stride, n, y, -100, temp, loss, lse, ws, wb, err, None)
    for bad in (dict(x=None), dict(x=FAKE + 1), dict(dt=lhs.LHS_F16), dict(dt=lhs.LHS_F32), dict(stride=63), dict(n=-1),
                dict(n=2 ** 24 + 1), dict(y=None), dict(y=FAKE + 2), dict(temp=0.0), dict(temp=-1.0), dict(temp=1e-45),
                dict(temp=float("nan")), dict(temp=float("inf")), dict(loss=None), dict(loss=FAKE + 2), dict(lse=None),
                dict(lse=FAKE + 1), dict(ws=None), dict(ws=FAKE + 128), dict(err=None), dict(err=FAKE + 2),
                dict(t=c_table(hidden=65544))):
        assert call(**bad) == lhs.LHS_ERR_INVALID_ARG, bad
    for dt in (lhs.LHS_F32, lhs.LHS_Q8_0):
        assert call(t=c_table(dt), dt=dt) == lhs.LHS_ERR_UNSUPPORTED
    assert call(n=0, x=None, y=None, loss=None, lse=None, ws=None, wb=0, err=None) == lhs.LHS_OK
    need = ctypes.c_size_t()
    assert L.lhs_loss_workspace(ctypes.byref(t), 5, ctypes.byref(need)) == 0 and need.value > 0
    assert call(wb=need.value - 1) == lhs.LHS_ERR_BUFFER_TOO_SMALL
    assert L.lhs_loss_workspace(ctypes.byref(t), -1, ctypes.byref(need)) == lhs.LHS_ERR_INVALID_ARG
    assert L.lhs_loss_workspace(ctypes.byref(t), 5, None) == lhs.LHS_ERR_INVALID_ARG
    assert L.lhs_loss_workspace(None, 5, ctypes.byref(need)) == lhs.LHS_ERR_INVALID_ARG


def test_grad_refuses():
    L, t = lhs.lib(), c_table()
    big, DW = 1 << 40, FAKE + 1000 * 64 * 2  # right behind the table

    def call(t=t, x=FAKE, dt=lhs.LHS_BF16, stride=64, n=5, y=FAKE, temp=1.0, lse=FAKE, dl=FAKE, dx=FAKE,
             dxt=lhs.LHS_BF16, dxs=64, dw=DW, dwt=lhs.LHS_BF16, acc=0, ws=FAKE, wb=big, err=FAKE):
        return L.lhs_loss_grad(ctypes.byref(t), x, dt, stride, n, y, -100, temp, lse, dl, dx, dxt, dxs, dw, dwt, acc, ws,
                               wb, err, None)
    for bad in (dict(x=None), dict(dt=lhs.LHS_F16), dict(stride=63), dict(n=-1), dict(n=2 ** 24 + 1), dict(y=None),
                dict(temp=0.0), dict(lse=None), dict(lse=FAKE + 2), dict(dl=None), dict(dl=FAKE + 2),
                dict(dx=None, dw=None), dict(dx=FAKE + 1), dict(dx=FAKE + 2, dxt=lhs.LHS_F32), dict(dxt=lhs.LHS_F16),
                dict(dxs=63), dict(dw=DW + 8), dict(dw=FAKE), dict(dw=DW - 16), dict(dw=FAKE - 16), dict(dwt=lhs.LHS_F16), dict(dwt=lhs.LHS_Q8_0), dict(acc=2),
                dict(acc=-1), dict(ws=None), dict(ws=FAKE + 16), dict(err=None)):
        assert call(**bad) == lhs.LHS_ERR_INVALID_ARG, bad
    assert call(t=c_table(lhs.LHS_F32), dt=lhs.LHS_F32) == lhs.LHS_ERR_UNSUPPORTED
    need = ctypes.c_size_t()
    assert L.lhs_loss_grad_workspace(ctypes.byref(t), 5, ctypes.byref(need)) == 0
    assert call(wb=need.value - 1) == lhs.LHS_ERR_BUFFER_TOO_SMALL
    # nothing to do: no positions, no table gradient to clear
    assert call(n=0, dw=None, dx=None, x=None, y=None, lse=None, dl=None, ws=None, wb=0, err=None) == lhs.LHS_OK
    assert call(n=0, acc=1, ws=None, wb=0) == lhs.LHS_OK


def test_bindings_refuse_cpu_tensors():
    x, y = torch.zeros((2, 8), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises((ValueError, AttributeError)):
        lhs.lhs_loss(None, x, y)
    with pytest.raises((ValueError, AttributeError)):
        lhs.lhs_loss_grad(None, x, y, torch.zeros(2), torch.zeros(2))


# ---------------------------------------------------------------------------
# the formulas in 64 bits, with the tolerances above
# ---------------------------------------------------------------------------
def grid_values(shape, g, step, most, dtype):
    """Multiples of step, up to most of them: sums of products are exact in f32."""
    return (torch.randint(-most, most + 1, shape, generator=g) * step).to(dtype)


def make(t, v, h, dtype, seed=0, exact=True, masked=0.2):
    g = torch.Generator().manual_seed(seed * 1000003 + t * 7919 + v * 31 + h)
    if exact:
        w = grid_values((v, h), g, 2.0 ** -6, 15, dtype)
        x = grid_values((t, h), g, 2.0 ** -4, 15, dtype)
        k = max(1, h // 256)
        x = (x.float() * (torch.arange(h) % k == 0)).to(dtype)  # logits of a few units
    else:
        w = (torch.randn((v, h), generator=g) * 0.05).to(dtype)
        x = (torch.randn((t, h), generator=g) * (10.0 / h ** 0.5)).to(dtype)
    y = torch.randint(0, v, (t,), generator=g, dtype=torch.int32)
    y[torch.rand(t, generator=g) < masked] = -100
    dl = torch.rand(t, generator=g) * 2 - 0.5
    return w.cuda(), x.cuda(), y.cuda(), dl.cuda()


def reference(w, x, y, dl, temp=1.0, exact=True, ignore=-100, outs=True):
    """Everything by the definition, and how far each may be off."""
    inv = float(torch.tensor(1.0 / temp, dtype=torch.float32)) if temp != 1.0 else 1.0
    v, h = w.shape
    on = (y >= 0) & (y < v) & (y != ignore)
    W, X, u = w.double(), x[on].double(), torch.finfo(w.dtype).eps / 2
    z = X @ W.T * inv
    # the temperature's inverse is rounded to f32
    dz = (2.0 ** -23 * z.abs().amax(1, keepdim=True) if temp != 1.0 else torch.zeros((len(X), 1), device=w.device, dtype=torch.float64))
    if not exact:
        dz = dz + h * 2.0 ** -23 * inv * (X.abs() @ W.abs().T).amax(1, keepdim=True)
    lse = torch.logsumexp(z, 1, keepdim=True)
    at = y[on].long()[:, None]
    loss = (lse - z.gather(1, at))[:, 0]
    r = {"on": on, "loss": loss, "lse": lse[:, 0],
         "tol": (2 * (E + dz) + 2.0 ** -22 * (lse.abs() + z.abs().amax(1, keepdim=True)))[:, 0]}
    if not outs:
        return r
    p = torch.exp(z - lse)
    hot = torch.zeros_like(p).scatter_(1, at, 1.0)
    d = dl[on].double()[:, None] * inv
    g = (p - hot) * d
    top = float(d.abs().max()) if len(d) else 0.0
    tiny = top * 2.0 ** -39 if w.dtype == torch.float16 else 0.0
    dg = u * g.abs() + 2 * (E + dz) * p * d.abs() + tiny
    r["dx"], r["dw"] = g @ W, g.T @ X
    r["dx_tol"] = dg @ W.abs() + v * 2.0 ** -23 * (g.abs() @ W.abs())
    r["dw_tol"] = dg.T @ X.abs() + (len(X) + 1) * 2.0 ** -23 * (g.abs().T @ X.abs())
    return r


def rounding(ref, dtype):
    e = torch.finfo(dtype).eps / 2
    return e * ref.abs() + (2.0 ** -25 if dtype == torch.float16 else 1e-40)


def within(got, ref, tol):
    d = (got.double() - ref).abs()
    assert got.shape == ref.shape
    worst = float((d / (tol + 1e-300)).max()) if d.numel() else 0.0
    assert bool((d <= tol).all()), f"{worst} of the tolerance"


def table_of(w):
    return lhs.lhs_table_init(w, *w.shape, CODE[w.dtype])


def check_loss(loss, lse, r):
    on = r["on"]
    assert bool((loss[~on] == 0).all()) and bool((lse[~on] == 0).all())
    within(loss[on], r["loss"], r["tol"])
    within(lse[on], r["lse"], r["tol"])


def check_grad(dx, dw, r, base=None):
    on = r["on"]
    if dx is not None:
        assert bool((dx[~on] == 0).all())
        within(dx[on], r["dx"], r["dx_tol"] + rounding(r["dx"], dx.dtype) * 1.01)
    if dw is not None:
        ref, extra = r["dw"], 0.0
        if base is not None:
            ref, extra = ref + base.double(), rounding(r["dw"], dw.dtype)
        within(dw, ref, r["dw_tol"] + extra + rounding(ref, dw.dtype) * 1.01)


SIZES = [(1, 1, 1), (1, 2, 8), (3, 7, 5), (1, 256, 64), (2, 257, 65), (5, 255, 63), (16, 8192, 256), (37, 1001, 1001),
         (64, 512, 128), (127, 300, 96), (128, 1000, 72), (129, 513, 200), (255, 600, 264), (256, 768, 256),
         (257, 1024, 896), (300, 9001, 40), (513, 2000, 513), (700, 300, 1030), (1100, 8191, 130), (2, 40000, 768),
         (40, 30011, 1544)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("t,v,h", SIZES)
def test_loss_sizes(t, v, h, dtype):
    w, x, y, dl = make(t, v, h, dtype)
    loss, lse, err = lhs.lhs_loss(table_of(w), x, y)
    assert int(err.item()) == 0
    check_loss(loss, lse, reference(w, x, y, dl, outs=False))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("t,v,h", SIZES)
def test_grad_sizes(t, v, h, dtype):
    w, x, y, dl = make(t, v, h, dtype)
    r = reference(w, x, y, dl)
    tab = table_of(w)
    _, lse, err = lhs.lhs_loss(tab, x, y)
    dx, dw, _ = lhs.lhs_loss_grad(tab, x, y, lse, dl, err=err)
    assert int(err.item()) == 0
    check_grad(dx, dw, r)


@pytest.mark.gpu
@pytest.mark.parametrize("temp", [1.0, 0.7, 3.0])
@pytest.mark.parametrize("dtype", HALF, ids=str)
def test_random_values_and_temperature(dtype, temp):
    w, x, y, dl = make(200, 3000, 320, dtype, exact=False)
    r = reference(w, x, y, dl, temp, exact=False)
    tab = table_of(w)
    loss, lse, err = lhs.lhs_loss(tab, x, y, temperature=temp)
    check_loss(loss, lse, r)
    dx, dw, _ = lhs.lhs_loss_grad(tab, x, y, lse, dl, temperature=temp, err=err)
    check_grad(dx, dw, r)
    assert int(err.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("h", [256, 100, 33])
@pytest.mark.parametrize("dtype", HALF, ids=str)
def test_outputs_of_both_types_added_and_alone(dtype, h):
    w, x, y, dl = make(150, 900, h, dtype)
    r = reference(w, x, y, dl)
    tab = table_of(w)
    _, lse, err = lhs.lhs_loss(tab, x, y)
    g = torch.Generator().manual_seed(h)
    for out in (dtype, torch.float32):
        wide = torch.full((150, h + 9), 7.0, dtype=out, device="cuda")
        dx = wide[:, 3:3 + h]
        dw = torch.full((900, h), float("nan"), dtype=out, device="cuda")
        lhs.lhs_loss_grad(tab, x, y, lse, dl, dx=dx, dtable=dw, err=err)
        check_grad(dx, dw, r)
        assert bool((wide[:, :3] == 7).all()) and bool((wide[:, 3 + h:] == 7).all())
        base = torch.randn((900, h), generator=g).to(out).cuda()
        both = base.clone()
        a, b, _ = lhs.lhs_loss_grad(tab, x, y, lse, dl, want_dx=False, dtable=both, accumulate=True, err=err)
        assert a is None and b is both
        check_grad(None, both, r, base)
        a, b, _ = lhs.lhs_loss_grad(tab, x, y, lse, dl, want_dtable=False, err=err)
        assert b is None
        check_grad(a, None, r)
    assert int(err.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("h", [64, 100, 257])
def test_strided_residuals(h):
    w, x, y, dl = make(300, 700, h, torch.bfloat16)
    r = reference(w, x, y, dl)
    for pad, off in ((8, 8), (3, 1), (5, 2)):  # aligned rows apart, and rows at any address
        wide = torch.full((300, h + pad + 8), float("nan"), dtype=x.dtype, device="cuda")
        xs = wide[:, off:off + h]
        xs.copy_(x)
        loss, lse, err = lhs.lhs_loss(table_of(w), xs, y)
        check_loss(loss, lse, r)
        dx, dw, _ = lhs.lhs_loss_grad(table_of(w), xs, y, lse, dl, err=err)
        check_grad(dx, dw, r)
        dx, dw, _ = lhs.lhs_loss_grad(table_of(w), xs, y, lse, dl, dx=xs, err=err)  # over the residuals
        check_grad(dx, dw, r)
        assert int(err.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("t", [1, 40, 600])
def test_positions_that_take_no_part(dtype, t):
    # whatever their residuals, lse and dloss hold, it reaches nothing
    w, x, y, dl = make(t, 1500, 136, dtype, masked=0.5)
    y[0] = -100
    if t > 8:
        y[3:7] = torch.tensor([-1, 1500, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    off = (y < 0) | (y >= 1500)
    r = reference(w, x, y, dl)
    x[off] = float("nan")
    if t > 20:
        x[off.nonzero()[5]] = float("inf")
    dl[off] = float("nan")
    tab = table_of(w)
    loss, lse, err = lhs.lhs_loss(tab, x, y)
    check_loss(loss, lse, r)
    want = lhs.LHS_ERRBIT_BAD_TOKEN if t > 8 else 0
    assert int(err.item()) == want
    lse[off] = float("nan")
    dx, dw, err = lhs.lhs_loss_grad(tab, x, y, lse, dl)
    assert int(err.item()) == want
    check_grad(dx, dw, r)
    # another id to ignore, inside the vocabulary
    y[:] = 7
    y[-1] = 9
    x[-1] = 0
    loss, lse, err = lhs.lhs_loss(tab, x, y, ignore=7)
    assert int(err.item()) == 0 and bool((loss[:-1] == 0).all())
    assert abs(float(loss[-1]) - torch.log(torch.tensor(1500.0)).item()) < 2 * E


@pytest.mark.gpu
@pytest.mark.parametrize("h", [64, 100])
def test_no_position_takes_part(h):
    w, x, y, dl = make(70, 700, h, torch.bfloat16)
    y[:] = -100
    x[:] = float("nan")
    tab = table_of(w)
    loss, lse, err = lhs.lhs_loss(tab, x, y)
    assert bool((loss == 0).all()) and bool((lse == 0).all())
    for out in (torch.bfloat16, torch.float32):
        dw = torch.full((700, h), float("nan"), dtype=out, device="cuda")
        dx, dw, _ = lhs.lhs_loss_grad(tab, x, y, lse, dl, dtable=dw, err=err)
        assert bool((dx == 0).all()) and bool((dw == 0).all())
        dw.fill_(3.0)
        lhs.lhs_loss_grad(tab, x, y, lse, dl, dtable=dw, accumulate=True, err=err)
        assert bool((dw == 3).all())
    # and no positions at all
    none = x[:0]
    loss, lse, _ = lhs.lhs_loss(tab, none, y[:0], err=err)
    assert loss.numel() == 0
    dw.fill_(3.0)
    dx, _, _ = lhs.lhs_loss_grad(tab, none, y[:0], lse, dl[:0], dtable=dw, accumulate=True, err=err)
    assert dx.shape == (0, h) and bool((dw == 3).all())
    lhs.lhs_loss_grad(tab, none, y[:0], lse, dl[:0], dtable=dw, err=err)
    assert bool((dw == 0).all()) and int(err.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF, ids=str)
def test_certain_and_hopeless_targets(dtype):
    # logits far apart: a target whose probability is 1 to f32, one whose is 0 to f32
    v, h = 600, 64
    w = torch.zeros((v, h), dtype=dtype, device="cuda")
    w[torch.arange(h), torch.arange(h)] = 1.0
    x = torch.zeros((4, h), dtype=dtype, device="cuda")
    x[0, 5], x[1, 5], x[2, 5], x[3, 5] = 100.0, 100.0, 20.0, -200.0
    y = torch.tensor([5, 6, 5, 5], dtype=torch.int32, device="cuda")
    dl = torch.ones(4, device="cuda")
    r = reference(w, x, y, dl)
    loss, lse, err = lhs.lhs_loss(table_of(w), x, y)
    check_loss(loss, lse, r)
    # log(1 + 599 exp(-d)): an exponential is good to 2^-21 and 2^-23 d log2(e) of its argument, a sum
    # of 599 to 2^-15 (the first form's 1 + s, which gave 0 for the first, lost what the second keeps)
    for k, d in ((0, 100.0), (2, 20.0)):
        want = math.log1p(599 * math.exp(-d))
        # exponentials below 2^-126 of the largest, as exp(-100) = 3.7e-44 is, may count as 0
        assert abs(float(loss[k]) - want) <= 2.0 ** -13 * want + 599 * 2.0 ** -126
    dx, dw, _ = lhs.lhs_loss_grad(table_of(w), x, y, lse, dl, err=err)
    check_grad(dx, dw, r)
    assert int(err.item()) == 0


@pytest.mark.gpu
def test_values_that_are_not_finite():
    w, x, y, dl = make(300, 900, 64, torch.bfloat16, masked=0.0)
    r = reference(w, x, y, dl)
    x[5, 3], x[260, 1] = float("nan"), float("inf")
    tab = table_of(w)
    loss, lse, err = lhs.lhs_loss(tab, x, y)
    assert int(err.item()) == lhs.LHS_ERRBIT_NONFINITE
    ok = torch.ones(300, dtype=torch.bool, device="cuda")
    ok[[5, 260]] = False
    assert bool(loss[~ok].isnan().all()) and bool(lse[~ok].isnan().all())
    within(loss[ok], r["loss"][ok], r["tol"][ok])
    dx, dw, err = lhs.lhs_loss_grad(tab, x, y, lse, dl)
    assert int(err.item()) == lhs.LHS_ERRBIT_NONFINITE
    assert bool(dx[~ok].isnan().all()) and bool(dw.isnan().all())
    within(dx[ok], r["dx"][ok], (r["dx_tol"] + rounding(r["dx"], dx.dtype) * 1.01)[ok])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF, ids=str)
def test_small_and_large_upstream_gradients(dtype):
    # f16 holds 2^-24 .. 65504: what the upstream gradient scales g to has to fit by itself
    w, x, y, dl = make(140, 2000, 72, dtype)
    tab = table_of(w)
    _, lse, err = lhs.lhs_loss(tab, x, y)
    for k in (2.0 ** -60, 2.0 ** -20, 2.0 ** 20, 2.0 ** 60):
        d = dl * k
        r = reference(w, x, y, d)
        dx = torch.empty(x.shape, device="cuda")
        dw = torch.empty(w.shape, device="cuda")
        lhs.lhs_loss_grad(tab, x, y, lse, d, dx=dx, dtable=dw, err=err)
        check_grad(dx, dw, r)
    d = torch.zeros_like(dl)
    dx, dw, _ = lhs.lhs_loss_grad(tab, x, y, lse, d, err=err)
    assert bool((dx == 0).all()) and bool((dw == 0).all()) and int(err.item()) == 0


@pytest.mark.gpu
def test_gradient_against_differences():
    """(L(+a) - L(-a)) / 2 along a direction, L = sum dloss * loss by the kernel, against the gradient
    along it.  A loss is off by 2E + its rounding, the third derivative of log sum exp along a direction
    in which the logits move by at most m is at most (2m)^3 / 10 (a third central moment of a variable in
    an interval of 2m), so the difference is off by a sixth of that, and the sum of the loss errors."""
    t, v, h = 24, 1000, 128
    w, x, y, _ = make(t, v, h, torch.bfloat16, masked=0.1)
    dl = torch.rand(t, generator=torch.Generator().manual_seed(1)).cuda() + 0.5
    on = (y >= 0).double()
    tab = table_of(w)

    def total(w, x):
        return float((lhs.lhs_loss(table_of(w), x, y)[0].double() * dl.double() * on).sum())
    _, lse, _ = lhs.lhs_loss(tab, x, y)
    dx32, dw32 = torch.empty(x.shape, device="cuda"), torch.empty(w.shape, device="cuda")
    lhs.lhs_loss_grad(tab, x, y, lse, dl, dx=dx32, dtable=dw32)
    r = reference(w, x, y, dl)
    noise = float((r["tol"] * dl[r["on"]].double()).sum())
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        for which in ("x", "w"):
            ref = x if which == "x" else w
            step = (2.0 ** -3 if which == "x" else 2.0 ** -5)
            d = ((torch.randint(0, 2, ref.shape, generator=g) * 2 - 1) * step).cuda()
            up, down = (ref.float() + d).to(ref.dtype), (ref.float() - d).to(ref.dtype)
            assert torch.equal(up.float() - down.float(), 2 * d)  # exact steps
            diff = (total(w, up) - total(w, down)) / 2 if which == "x" else (total(up, x) - total(down, x)) / 2
            grad = float(((dx32 if which == "x" else dw32).double() * d.double()).sum())
            move = (d.double() @ w.double().T if which == "x" else x.double() @ d.double().T).abs().amax(1)
            curve = float(((2 * move) ** 3 / 60 * dl.double() * on).sum())
            slack = float((r["dx_tol"].sum() if which == "x" else r["dw_tol"].sum())) * step
            assert abs(diff - grad) <= curve + noise + slack, (which, diff, grad)


@pytest.mark.gpu
@pytest.mark.parametrize("t,v,h", [(300, 5000, 264), (1000, 70000, 64)])
def test_runs_are_alike(t, v, h):
    w, x, y, dl = make(t, v, h, torch.bfloat16, exact=False)
    tab = table_of(w)
    first = None
    for _ in range(5):
        loss, lse, _ = lhs.lhs_loss(tab, x, y)
        dx, dw, _ = lhs.lhs_loss_grad(tab, x, y, lse, dl)
        if first is None:
            first = [loss, lse, dx, dw]
        assert all(torch.equal(a, b) for a, b in zip(first, [loss, lse, dx, dw]))


@pytest.mark.gpu
def test_captured_calls_replay():
    # the number of positions that take part may differ from the one captured
    t, v, h = 520, 3000, 136
    w, x, y, dl = make(t, v, h, torch.bfloat16)
    tab = table_of(w)
    ws = torch.empty(lhs.lhs_loss_workspace(tab, t), dtype=torch.uint8, device="cuda")
    gws = torch.empty(lhs.lhs_loss_grad_workspace(tab, t), dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        lhs.lhs_loss(tab, x, y, loss=loss, lse=lse, ws=ws, err=err)
        lhs.lhs_loss_grad(tab, x, y, lse, dl, dx=dx, dtable=dw, ws=gws, err=err)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        w2, x2, y2, dl2 = make(t, v, h, torch.bfloat16, seed=seed + 1, masked=0.3 * seed)
        for a, b in ((w, w2), (x, x2), (y, y2), (dl, dl2)):
            a.copy_(b)
        ws.fill_(0xFF)
        gws.fill_(0xFF)
        graph.replay()
        r = reference(w, x, y, dl)
        check_loss(loss, lse, r)
        check_grad(dx, dw, r)
    assert int(err.item()) == 0


@pytest.mark.gpu
def test_streams():
    # two streams at once, each with buffers of its own; what a call allocates itself too
    t, v, h = 400, 20000, 256
    data = [make(t, v, h, torch.bfloat16, seed=s) for s in range(2)]
    refs = [reference(*d) for d in data]
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        torch.cuda._sleep(5_000_000)  # the current stream gets to nothing meanwhile
        got = []
        for k in range(2):
            w, x, y, dl = data[k]
            loss, lse, err = lhs.lhs_loss(table_of(w), x, y, stream=st[k])
            dx, dw, _ = lhs.lhs_loss_grad(table_of(w), x, y, lse, dl, err=err, stream=st[k].cuda_stream)
            got.append((loss, lse, dx, dw, err))
        torch.cuda.synchronize()
        for k in range(2):
            check_loss(got[k][0], got[k][1], refs[k])
            check_grad(got[k][2], got[k][3], refs[k])
            assert int(got[k][4].item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("h", [256, 100])
def test_nothing_else_is_written(h):
    from gpu_util import canaries_intact, guarded
    w, x, y, dl = make(90, 777, h, torch.bfloat16)
    tab = table_of(w)
    need, gneed = lhs.lhs_loss_workspace(tab, 90), lhs.lhs_loss_grad_workspace(tab, 90)
    bufs = [guarded((n,), dt) for n, dt in ((90, torch.float32), (90, torch.float32), (need, torch.uint8),
                                            (gneed, torch.uint8))]
    loss, lse, ws, gws = [b[1] for b in bufs]
    outs = [guarded((90, h), torch.bfloat16), guarded((777, h), torch.bfloat16)]
    bufs += outs
    lhs.lhs_loss(tab, x, y, loss=loss, lse=lse, ws=ws)
    lhs.lhs_loss_grad(tab, x, y, lse, dl, dx=outs[0][1], dtable=outs[1][1], ws=gws)
    check_grad(outs[0][1], outs[1][1], reference(w, x, y, dl))
    assert all(canaries_intact(raw, pad) for raw, _, pad in bufs)


@pytest.mark.gpu
def test_offsets_pass_32_bits():
    # the table's elements and its gradient's lie beyond 2^31
    v, h, t = 3_000_000, 768, 40
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    w = torch.zeros((v, h), dtype=torch.bfloat16, device="cuda")
    w[-1, 0], w[-2, 1], w[-300, 2] = 4.0, 8.0, 2.0
    x = torch.zeros((t, h), dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[1, 1], x[2, 2] = 4.0, 2.0, 9.0
    y = torch.full((t,), v - 1, dtype=torch.int32, device="cuda")
    y[1], y[2], y[3] = v - 2, v - 300, 0
    dl = torch.ones(t, device="cuda")
    tab = table_of(w)
    loss, lse, err = lhs.lhs_loss(tab, x, y)
    z = torch.zeros((t, 4), dtype=torch.float64)
    for k, (row, col) in enumerate(((v - 1, 0), (v - 2, 1), (v - 300, 2))):
        z[:, k] = float(w[row, col]) * x[:, col].double().cpu()
    n = torch.logsumexp(torch.cat([z[:, :3], torch.full((t, 1), float(torch.log(torch.tensor(v - 3.0))), dtype=torch.float64)], 1), 1)
    at = torch.tensor([0] + [1, 2, 3] + [0] * (t - 4))
    want = n - z.gather(1, at[:, None])[:, 0]
    assert float((loss.cpu().double() - want).abs().max()) < 2 * E * 8  # V < 2^22: 12,000 more additions of 2^-24
    dx, dw, _ = lhs.lhs_loss_grad(tab, x, y, lse, dl, err=err)
    assert int(err.item()) == 0
    p = torch.exp(z[:, :3] - n[:, None])
    g = p.clone()
    for i in range(3):
        g[at == i, i] -= 1.0
    wantw = g.T @ x.double().cpu()
    got = dw[[v - 1, v - 2, v - 300]].double().cpu()
    assert float((got - wantw).abs().max()) <= 2.0 ** -7 * float(wantw.abs().max())
    assert float((dw[0, 0].double().cpu() - (float(torch.exp(-n[3])) * 4 - 4 + 4 * float(torch.exp(-n).sum() - torch.exp(-n[3])))).abs()) <= 2.0 ** -6
