"""Sampling: refusals, and draws against the definition in 64 bits.

The kernel's weights are good to about 2^-36 of themselves (2^-35 is granted
below), so the running sums and filter borders are too.  Where the definition,
in 64 bits, comes closer than 2^-33 of the total to a border (of top-p,
min-p or the draw), the row says nothing and is skipped; elsewhere the token
has to be the same.  The probability is one binary32 rounding (2^-24) of a
quotient good to 2^-34: 2^-23 covers it.
"""
import math

import numpy as np
import pytest
import torch

import embedding_lookup_tied_gb300 as lhs

FAKE = 0x10000
NEAR = 2.0 ** -33
WIDE = [torch.float32, torch.float16, torch.bfloat16]


def test_refuses():
    L = lhs.lib()

    def call(x=FAKE, dt=0, stride=100, rows=2, v=100, u=FAKE, t=None, k=None, p=None, m=None, ids=FAKE, pr=None,
             err=FAKE):
        return L.lhs_sample(x, dt, stride, rows, v, u, t, k, p, m, ids, pr, err, None)
    for bad in (dict(x=None), dict(x=FAKE + 2), dict(x=FAKE + 1, dt=1), dict(dt=lhs.LHS_Q8_0), dict(dt=-1),
                dict(stride=99), dict(rows=-1), dict(rows=2 ** 31), dict(v=0), dict(v=2 ** 31, stride=2 ** 31),
                dict(u=None), dict(u=FAKE + 2), dict(t=FAKE + 1), dict(k=FAKE + 2), dict(p=FAKE + 3),
                dict(m=FAKE + 2), dict(ids=None), dict(ids=FAKE + 2), dict(pr=FAKE + 2), dict(err=None)):
        assert call(**bad) == lhs.LHS_ERR_INVALID_ARG, bad
    assert call(rows=0, x=None, u=None, ids=None, err=None) == lhs.LHS_OK


def test_binding_refuses():
    with pytest.raises(ValueError):
        lhs.lhs_sample(torch.zeros((2, 8)), torch.zeros(2))


def reference(row, u, t=1.0, k=0, p=1.0, q=0.0):
    """(token, probability, whether a border is too near to tell) by the
    definition.  row: float64; the parameters as the binary32 numbers given."""
    v = len(row)
    t, k = (1.0, 1) if t == 0 else (min(max(t, 2.0 ** -100), 2.0 ** 100), k)
    with np.errstate(over="ignore", invalid="ignore"):
        w = np.exp((row - row.max()) / t)
    order = np.argsort(-row, kind="stable")
    if 0 < k < v:
        order = order[:k]
    near = False
    ws = w[order]
    if p < 1:
        c = np.cumsum(ws)
        n = int(np.searchsorted(c, p * c[-1], side="left")) + 1
        near |= bool(np.min(np.abs(c / c[-1] - p)) < NEAR)
        order, ws = order[:n], ws[:n]
    if q > 0:
        near |= bool(np.any(np.abs(ws - q) < NEAR * q)) and q < 1
        order = order[ws >= q]
    ids = np.sort(order)
    c = np.cumsum(w[ids])
    at = int(np.searchsorted(c, u * c[-1], side="right"))
    near |= bool(np.min(np.abs(c / c[-1] - u)) < NEAR) and len(ids) > 1 and u > 0
    tok = int(ids[at])
    return tok, w[tok] / c[-1], near


def check(logits, u, t=None, k=None, p=None, q=None, most_skipped=0.02, **kw):
    """Every row of lhs_sample against reference().  Arguments: CPU tensors."""
    n = logits.shape[0]
    up = lambda a: None if a is None else a.cuda()  # noqa: E731
    dev = kw.pop("device_logits", None)
    ids, probs, err = lhs.lhs_sample(logits.cuda() if dev is None else dev, up(u), up(t), up(k), up(p), up(q), **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    ids, probs = ids.cpu().tolist(), probs.cpu().numpy().astype(np.float64)
    rows = logits.double().numpy()
    get = lambda a, r, off: off if a is None else float(a[r])  # noqa: E731
    skipped = 0
    for r in range(n):
        tok, pr, near = reference(rows[r], float(u[r]), get(t, r, 1.0), int(get(k, r, 0)), get(p, r, 1.0),
                                  get(q, r, 0.0))
        if near:
            skipped += 1
            continue
        assert ids[r] == tok, (r, ids[r], tok)
        assert abs(probs[r] - pr) <= 2.0 ** -23 * pr, (r, probs[r], pr)
    assert skipped <= max(1, most_skipped * n)


def draw_rows(seed, n, v, dtype=torch.float32, spread=(0.5, 5.0)):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, v), generator=g) * (torch.rand((n, 1), generator=g) * (spread[1] - spread[0]) + spread[0])
    return x.to(dtype), torch.rand(n, generator=g), g


def params(g, n, v, mode):
    t = torch.rand(n, generator=g) * 1.5 + 0.3
    k = torch.randint(1, max(2, min(v, 200)), (n,), generator=g, dtype=torch.int32) if mode in ("k", "all") else None
    p = torch.rand(n, generator=g) * 0.6 + 0.39 if mode in ("p", "all") else None
    q = torch.rand(n, generator=g) * 0.2 if mode in ("q", "all") else None
    if mode == "all":
        off = torch.randint(0, 8, (n,), generator=g)
        k[off % 2 == 0] = 0
        p[off == 3] = 1.0
        q[off >= 4] = 0.0
        t[off == 7] = 0.0
    return t, k, p, q


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", WIDE, ids=str)
@pytest.mark.parametrize("mode", ["none", "k", "p", "q", "all"])
@pytest.mark.parametrize("n,v", [(40, 1), (40, 2), (40, 31), (30, 33), (64, 100), (48, 511), (24, 1000), (40, 8191),
                                 (20, 16384), (6, 50001)])
def test_draws(dtype, mode, n, v):
    x, u, g = draw_rows(n * 1000 + v, n, v, dtype)
    t, k, p, q = params(g, n, v, mode)
    check(x, u, t, k, p, q)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["none", "p", "all"])
@pytest.mark.parametrize("v,dtype", [(151936, torch.float32), (262144, torch.bfloat16), (262145, torch.float32),
                                     (600001, torch.float16), (800001, torch.float32),
                                     (1200003, torch.float32)])
def test_long_rows(mode, v, dtype):
    x, u, g = draw_rows(v, 3, v, dtype)
    t, k, p, q = params(g, 3, v, mode)
    check(x, u, t, k, p, q)


@pytest.mark.gpu
@pytest.mark.parametrize("v", [50, 3001, 70000])
def test_many_draws_of_one_row(v):
    # a grid of random numbers over one row walks its whole running sum
    x, _, _ = draw_rows(7, 1, v)
    n = 400
    u = (torch.arange(n) + 0.5) / n
    u[0], u[1] = 0.0, 1.0 - 2.0 ** -24
    check(x.expand(n, v).contiguous(), u, p=torch.full((n,), 0.9), t=torch.full((n,), 0.7))


@pytest.mark.gpu
@pytest.mark.parametrize("v", [64, 5000, 40000])
def test_many_rows(v):
    n = 700
    x, u, g = draw_rows(v, n, v)
    t, k, p, q = params(g, n, v, "all")
    check(x, u, t, k, p, q)


@pytest.mark.gpu
def test_more_rows_than_one_grid():
    # more rows than CTAs: each works through several, at changing alignments
    n, v = (1 << 20) + 4321, 7
    x, u, _ = draw_rows(4, n, v)
    xd, ud = x.cuda(), u.cuda()
    k = torch.full((n,), 3, dtype=torch.int32, device="cuda")
    for args in (dict(), dict(top_k=k)):
        ids, probs, err = lhs.lhs_sample(xd, ud, **args)
        assert int(err.item()) == 0
        w = torch.exp(x.double() - x.double().amax(1, keepdim=True))
        if args:
            w = torch.where(x >= x.topk(3, dim=1).values[:, -1:], w, 0.0)
        c = w.cumsum(1)
        share = c / c[:, -1:]
        far = (share - u.double()[:, None]).abs().amin(1) > NEAR
        want = (share <= u.double()[:, None]).sum(1)
        assert int(far.sum()) > 0.99 * n
        assert torch.equal(ids.cpu()[far].long(), want[far])


@pytest.mark.gpu
@pytest.mark.parametrize("v", [10, 4096, 30000, 262144])
def test_equal_logits(v):
    # ties: lower ids first.  Powers of two make every share exact.
    n = 6
    x = torch.zeros((n, v))
    u = torch.tensor([0.0, 0.3, 0.6, 0.9, 0.99, 0.5])
    k = torch.tensor([1, 2, 3, 7, v, 5], dtype=torch.int32)
    ids, probs, _ = lhs.lhs_sample(x.cuda(), u.cuda(), top_k=k.cuda())
    kk = k.double()
    assert ids.cpu().tolist() == [int(math.floor(float(u[r]) * float(kk[r]))) for r in range(n)]
    assert torch.allclose(probs.cpu().double(), 1 / kk, rtol=2.0 ** -23, atol=0)
    # top-p over equal weights keeps ceil(p v) of them
    p = torch.tensor([0.5, 0.25, 0.75, 2.0 ** -20, 1.0, 0.125])
    ids, probs, _ = lhs.lhs_sample(x.cuda(), u.cuda(), top_p=p.cuda())
    kept = [math.ceil(float(p[r]) * v) for r in range(n)]
    assert torch.allclose(probs.cpu().double(), 1 / torch.tensor(kept).double(), rtol=2.0 ** -23, atol=0)
    for r in range(n):
        assert abs(int(ids[r]) - float(u[r]) * kept[r]) <= 1 and int(ids[r]) < kept[r]
    # a few levels, most rows in ties, every filter at once
    g = torch.Generator().manual_seed(v)
    y = torch.randint(0, 4, (40, v), generator=g).float()
    t, k, p, q = params(g, 40, v, "all")
    check(y, torch.rand(40, generator=g), t, k, p, None)


@pytest.mark.gpu
@pytest.mark.parametrize("v", [40, 9000, 100000])
def test_greedy(v):
    x, u, _ = draw_rows(v, 8, v)
    x[1, v // 3:v // 3 + 3] = 50.0  # equal largest: the lowest id
    x[2] = float("-inf")
    x[2, v - 1] = -3.0
    x[3] = -torch.finfo(torch.float32).max
    x[4, 0] = x[4].max()
    t = torch.zeros(8)
    p = torch.full((8,), 0.5)
    ids, probs, err = lhs.lhs_sample(x.cuda(), u.cuda(), t.cuda(), top_p=p.cuda())
    assert int(err.item()) == 0
    assert ids.cpu().tolist() == x.argmax(1).tolist() and ids[3] == 0 and ids[4] == 0
    assert bool((probs == 1).all())


@pytest.mark.gpu
@pytest.mark.parametrize("v", [33, 5000, 150000])
def test_masks(v):
    x, u, g = draw_rows(v, 12, v)
    mask = torch.rand((12, v), generator=g) < 0.95
    mask[:, v // 2] = False
    x.masked_fill_(mask, float("-inf"))
    x[3:6].masked_fill_(mask[3:6], torch.finfo(torch.float32).min)  # the type's lowest value
    x[6] = float("-inf")
    x[6, v - 2] = 1.5  # one token left
    x[7] = torch.finfo(torch.float32).min  # nothing but lowest values: all alike
    x[8] = float("-inf")
    x[8, :2] = torch.tensor([torch.finfo(torch.float32).max, torch.finfo(torch.float32).min])
    t, k, p, q = params(g, 12, v, "all")
    check(x, u, t, k, p, q)
    check(x, u, p=torch.full((12,), 0.7))
    check(x, u, k=torch.full((12,), 30, dtype=torch.int32))
    check(x, u)


@pytest.mark.gpu
@pytest.mark.parametrize("v", [20, 6000, 200000])
def test_rows_without_an_answer(v):
    x, u, _ = draw_rows(v, 14, v)
    t, p, q = torch.ones(14), torch.full((14,), 0.9), torch.full((14,), 0.01)
    x[1] = float("-inf")

    def bits(keep):
        rows = [0] + keep
        ids, probs, err = lhs.lhs_sample(x[rows].cuda(), u[rows].cuda(), t[rows].cuda(), None, p[rows].cuda(),
                                         q[rows].cuda())
        assert int(ids[0]) >= 0 and float(probs[0]) > 0
        assert ids[1:].tolist() == [-1] * len(keep) and probs[1:].tolist() == [0] * len(keep)
        return int(err.item())
    assert bits([1]) == 0  # nothing left by the mask: no error
    x[2, v // 2] = float("nan")
    x[3, v - 1] = float("inf")
    x[4] = float("-inf")
    x[4, 0] = -float("nan")
    for r in (2, 3, 4):
        assert bits([r]) == lhs.LHS_ERRBIT_NONFINITE
    t[5], t[6], t[7] = -0.5, float("inf"), float("nan")
    p[8], p[9] = 0.0, 1.5
    q[10], q[11] = -0.1, 1.01
    u[12], u[13] = 1.0, -0.25
    for r in range(5, 14):
        assert bits([r]) == lhs.LHS_ERRBIT_BAD_PARAM, r
    assert bits([2, 9]) == lhs.LHS_ERRBIT_NONFINITE | lhs.LHS_ERRBIT_BAD_PARAM


@pytest.mark.gpu
def test_extreme_parameters():
    v = 3000
    x, u, _ = draw_rows(5, 10, v)
    f = torch.float32
    t = torch.tensor([1e-30, 1e-3, 1e4, 1e30, 1.0, 1.0, 1.0, 1.0, 3e38, 1e-38], dtype=f)
    k = torch.tensor([0, 0, 0, 0, -1, v, v + 5, v - 1, 0, 0], dtype=torch.int32)
    p = torch.tensor([1, 1, 1, 1, 1e-30, 1 - 2.0 ** -24, 0.5, 1, 1, 0.3], dtype=f)
    q = torch.tensor([0, 0, 0, 0, 0, 0, 1.0, 1e-30, 0, 0], dtype=f)
    check(x, u, t, k, p, q)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", WIDE, ids=str)
@pytest.mark.parametrize("v", [63, 1001, 20000, 140001])
def test_strides_alignment_and_canaries(dtype, v):
    n = 9
    x, u, g = draw_rows(v, n, v, dtype)
    t, k, p, q = params(g, n, v, "all")
    for off in (1, 3, 8):
        big = torch.full((n, v + 29), float("nan"), dtype=dtype, device="cuda")  # NaN between the rows: never read
        big[:, off:off + v] = x.cuda()
        before = big.clone()
        check(x, u, t, k, p, q, device_logits=big[:, off:off + v])
        assert torch.equal(big.view(torch.uint8), before.view(torch.uint8))


@pytest.mark.gpu
def test_results_repeat():
    # integer sums: the same bits every time
    x, u, g = draw_rows(3, 60, 100000)
    t, k, p, q = params(g, 60, 100000, "p")
    args = [a.cuda() if a is not None else None for a in (x, u, t, k, p, q)]
    first = lhs.lhs_sample(*args)
    for _ in range(5):
        again = lhs.lhs_sample(*args)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.gpu
def test_no_probs_no_rows_other_stream():
    x, u, _ = draw_rows(1, 5, 777)
    ids, probs, _ = lhs.lhs_sample(x.cuda(), u.cuda(), want_probs=False)
    assert probs is None
    st = torch.cuda.Stream()
    xd, ud = x.cuda(), u.cuda()
    torch.cuda.synchronize()
    other, _, _ = lhs.lhs_sample(xd, ud, err=torch.zeros(1, dtype=torch.int32, device="cuda"), stream=st)
    st.synchronize()
    assert torch.equal(ids, other)
    e, _, _ = lhs.lhs_sample(torch.empty((0, 777), device="cuda"), torch.empty(0, device="cuda"))
    assert e.numel() == 0


@pytest.mark.gpu
def test_captured_call_replays():
    v = 30000
    x, u, g = draw_rows(2, 16, v)
    t, k, p, q = params(g, 16, v, "all")
    xd, ud = x.cuda(), u.cuda()
    args = [a.cuda() for a in (t, k, p, q)]
    ids = torch.empty(16, dtype=torch.int32, device="cuda")
    probs = torch.empty(16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lhs.lhs_sample(xd, ud, *args, ids=ids, probs=probs, err=err)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        lhs.lhs_sample(xd, ud, *args, ids=ids, probs=probs, err=err)
    for seed in (11, 12):
        xn, un, _ = draw_rows(seed, 16, v)
        xd.copy_(xn)
        ud.copy_(un)
        gr.replay()
        again, pr, _ = lhs.lhs_sample(xn.cuda(), un.cuda(), *args)
        assert torch.equal(ids, again) and torch.equal(probs, pr)


@pytest.mark.gpu
def test_chained_after_the_product():
    # logits written by the product, then drawn from, on one stream
    rng = np.random.default_rng(1)
    n, k, m = 9000, 320, 7
    codes = torch.from_numpy(rng.integers(-127, 128, (n, k), dtype=np.int8)).cuda()
    tab = lhs.lhs_i8_init(codes, torch.full((n,), 1e-3, device="cuda"), k)
    x = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32)).cuda()
    u = torch.from_numpy(rng.random(m).astype(np.float32)).cuda()
    p = torch.full((m,), 0.9, device="cuda")
    out = torch.empty((m, n), device="cuda")
    ref = lhs.lhs_i8_logits(tab, x)[0]
    torch.cuda.synchronize()
    want = lhs.lhs_sample(ref, u, top_p=p)[0]
    for _ in range(50):
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        lhs.lhs_i8_logits(tab, x, out=out)
        assert torch.equal(lhs.lhs_sample(out, u, top_p=p)[0], want)
