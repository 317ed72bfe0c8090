"""The cross entropy's gradient where its products go through many pieces of the
vocabulary, splits and blocks of tokens, for equality.

The residuals and the table share no column in which both are other than 0, so
that every logit is 0; with lse = 5 ln 2 given, every probability is 2^-5 (the
kernel's, good to 2^-20, rounds to it in either type).  g = (2^-5 - [v = y])
dloss is then held exactly in bf16 and f16 where dloss is a power of two, and
both gradients are sums of multiples of one power of two that stay below 2^24 of
it: every order of sums gives the same bits.
"""
import math

import pytest
import torch

import embedding_lookup_tied_gb300 as lhs
from test_loss import check_grad, check_loss, make, reference, table_of, within

pytestmark = pytest.mark.gpu

HALF = [torch.bfloat16, torch.float16]


def flat(t, v, h, dtype, seed=0, masked=0.1):
    """(table, residuals, targets, lse, dloss) as above, and both gradients."""
    g = torch.Generator().manual_seed(seed + t * 31 + v * 7 + h)
    half = (torch.arange(h) % 2 == 0).float()
    w = torch.randint(-7, 8, (v, h), generator=g).float() * half / 8
    x = torch.randint(-7, 8, (t, h), generator=g).float() * (1 - half) / 8
    if h == 1:
        x = torch.zeros((t, 1))
    y = torch.randint(0, v, (t,), generator=g, dtype=torch.int32)
    y[torch.rand(t, generator=g) < masked] = -100
    dl = 2.0 ** torch.randint(-2, 1, (t,), generator=g).float()
    w, x, y, dl = w.cuda(), x.cuda(), y.cuda(), dl.cuda()
    on = y >= 0
    d = dl.double() * on
    dx = d[:, None] * (2.0 ** -5 * w.double().sum(0)[None, :] - w.double()[y.clamp(min=0).long()])
    xd = x.double() * d[:, None]
    dw = (2.0 ** -5 * xd.sum(0))[None, :].repeat(v, 1).index_add_(0, y.clamp(min=0).long(), -xd)
    lse = torch.full((t,), 5 * math.log(2), device="cuda")
    return w.to(dtype), x.to(dtype), y, lse, dl, dx, dw


# (tokens, vocabulary, hidden): several pieces, whole and ragged last ones, splits of dx, odd rows
SIZES = [(1, 100003, 64), (1, 180000, 200), (130, 90001, 72), (256, 262144, 16), (300, 60000, 320), (513, 50021, 40),
         (1500, 30011, 136), (2049, 20000, 264), (5000, 9000, 48), (20000, 2100, 24), (9000, 700, 520),
         (260, 80000, 33), (700, 41001, 101), (3000, 12345, 7), (70000, 300, 16), (4, 400003, 8), (30, 700, 9000), (600, 300, 20008)]


@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("t,v,h", SIZES)
def test_sums_are_exact(t, v, h, dtype):
    w, x, y, lse, dl, rx, rw = flat(t, v, h, dtype)
    tab = table_of(w)
    dx = torch.full((t, h), float("nan"), device="cuda")
    dw = torch.full((v, h), float("nan"), device="cuda")
    _, _, err = lhs.lhs_loss_grad(tab, x, y, lse, dl, dx=dx, dtable=dw)
    assert torch.equal(dx, rx.float()) and torch.equal(dw, rw.float())
    lhs.lhs_loss_grad(tab, x, y, lse, dl, want_dx=False, dtable=dw, accumulate=True, err=err)
    assert torch.equal(dw, 2 * rw.float())
    half, _, _ = lhs.lhs_loss_grad(tab, x, y, lse, dl, want_dtable=False, err=err)
    assert torch.equal(half, rx.float().to(dtype))
    _, half, _ = lhs.lhs_loss_grad(tab, x, y, lse, dl, want_dx=False, err=err)
    assert torch.equal(half, rw.float().to(dtype))
    base = torch.full((v, h), 3.0, dtype=dtype, device="cuda")
    lhs.lhs_loss_grad(tab, x, y, lse, dl, dtable=base, accumulate=True, err=err)
    assert torch.equal(base, (rw + 3).float().to(dtype))  # one rounding of the sum
    assert int(err.item()) == 0


@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("t,v,h", [(300, 60000, 72), (1500, 30011, 136), (600, 45000, 33), (2, 150000, 64)])
def test_pieces_against_the_formula(t, v, h, dtype):
    w, x, y, dl = make(t, v, h, dtype)
    r = reference(w, x, y, dl)
    tab = table_of(w)
    loss, lse, err = lhs.lhs_loss(tab, x, y)
    check_loss(loss, lse, r)
    dx, dw, _ = lhs.lhs_loss_grad(tab, x, y, lse, dl, err=err)
    check_grad(dx, dw, r)
    assert int(err.item()) == 0


@pytest.mark.parametrize("dtype", HALF, ids=str)
@pytest.mark.parametrize("t,v,h", [(1, 600, 64), (3, 40000, 72), (64, 8192, 256), (128, 3000, 33), (140, 100, 200)])
def test_few_positions_keep_g_in_two_terms(t, v, h, dtype):
    """Up to 128 positions that take part (of 140, a fifth does not): g is off by eps / 2 of eps / 2
    of itself; the rest as in test_loss."""
    w, x, y, dl = make(t, v, h, dtype, masked=0.2)
    r = reference(w, x, y, dl)
    on = r["on"]
    assert int(on.sum()) <= 128
    u = torch.finfo(dtype).eps / 2
    W, X, d = w.double(), x[on].double(), dl[on].double()[:, None]
    p = torch.exp(X @ W.T - r["lse"][:, None])
    g = (p - torch.zeros_like(p).scatter_(1, y[on].long()[:, None], 1.0)) * d
    dg = (u * u + 2.0 ** -22) * g.abs() + 2 * 2.0 ** -14 * p * d.abs() + (float(d.abs().max()) if len(d) else 0.0) * 2.0 ** -39
    tab = table_of(w)
    _, lse, err = lhs.lhs_loss(tab, x, y)
    dx, dw = torch.empty((t, h), device="cuda"), torch.empty((v, h), device="cuda")
    lhs.lhs_loss_grad(tab, x, y, lse, dl, dx=dx, dtable=dw, err=err)
    within(dx[on], r["dx"], dg @ W.abs() + v * 2.0 ** -23 * (g.abs() @ W.abs()))
    within(dw, r["dw"], dg.T @ X.abs() + 260 * 2.0 ** -23 * (g.abs().T @ X.abs()))
    assert bool((dx[~on] == 0).all()) and int(err.item()) == 0


@pytest.mark.parametrize("t,v,h", [(300, 60000, 320), (1500, 30011, 136)])
def test_several_at_once(t, v, h):
    # four calls on four streams, whose CTAs share the chip in whatever way: none waits for one that
    # does not run
    data = [flat(t, v, h, torch.bfloat16, seed=s) for s in range(4)]
    tabs = [table_of(d[0]) for d in data]
    st = [torch.cuda.Stream() for _ in range(4)]
    bufs = [(torch.empty((t, h), device="cuda"), torch.empty((v, h), device="cuda"),
             torch.empty(lhs.lhs_loss_grad_workspace(tabs[0], t), dtype=torch.uint8, device="cuda"),
             torch.zeros(1, dtype=torch.int32, device="cuda")) for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(6):
        for k in range(4):
            _, x, y, lse, dl = data[k][:5]
            dx, dw, ws, err = bufs[k]
            lhs.lhs_loss_grad(tabs[k], x, y, lse, dl, dx=dx, dtable=dw, ws=ws, err=err, stream=st[k])
        torch.cuda.synchronize()
        for k in range(4):
            dx, dw, _, err = bufs[k]
            assert int(err.item()) == 0
            assert torch.equal(dx, data[k][5].float()) and torch.equal(dw, data[k][6].float())
            dx.fill_(float("nan"))
            dw.fill_(float("nan"))


@pytest.mark.parametrize("t,v,h", [(6000, 30000, 8), (300, 400003, 16), (2000, 60001, 64)])
def test_items_handed_over_as_fast_as_they_can(t, v, h):
    # one stage of k to a tile of logits and one tile of columns: the items' slots are written again
    # as soon as the last of the roles has read them
    w, x, y, lse, dl, rx, rw = flat(t, v, h, torch.bfloat16)
    tab = table_of(w)
    ws = torch.empty(lhs.lhs_loss_grad_workspace(tab, t), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty((t, h), device="cuda"), torch.empty((v, h), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(20):
        dx.fill_(float("nan"))
        dw.fill_(float("nan"))
        lhs.lhs_loss_grad(tab, x, y, lse, dl, dx=dx, dtable=dw, ws=ws, err=err)
        assert torch.equal(dx, rx.float()) and torch.equal(dw, rw.float())
    assert int(err.item()) == 0


@pytest.mark.parametrize("t,v,h", [(3000, 60000, 520), (1025, 200000, 40)])
def test_slots_of_g_are_overwritten_after_their_last_reader(t, v, h):
    # more pieces than slots; dx's and dtable's tiles read a slot at their own pace, for one of the
    # two products, the other and both
    w, x, y, lse, dl, rx, rw = flat(t, v, h, torch.float16)
    tab = table_of(w)
    dx, dw = torch.empty((t, h), device="cuda"), torch.empty((v, h), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for k in range(12):
        dx.fill_(float("nan"))
        dw.fill_(float("nan"))
        lhs.lhs_loss_grad(tab, x, y, lse, dl, dx=dx, dtable=dw, want_dx=k % 3 != 1, want_dtable=k % 3 != 2, err=err)
        assert k % 3 == 1 or torch.equal(dx, rx.float())
        assert k % 3 == 2 or torch.equal(dw, rw.float())
    assert int(err.item()) == 0


def test_captured_with_other_numbers_of_positions():
    # the tiles of a captured call follow the positions that take part at its replay
    t, v, h = 1200, 40000, 72
    w, x, y, lse, dl, rx, rw = flat(t, v, h, torch.float16)
    tab = table_of(w)
    ws = torch.empty(lhs.lhs_loss_grad_workspace(tab, t), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty((t, h), device="cuda"), torch.empty((v, h), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lhs.lhs_loss_grad(tab, x, y, lse, dl, dx=dx, dtable=dw, ws=ws, err=err)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lhs.lhs_loss_grad(tab, x, y, lse, dl, dx=dx, dtable=dw, ws=ws, err=err)
    for seed, masked in enumerate((0.0, 0.3, 0.9, 1.1)):
        new = flat(t, v, h, torch.float16, seed=seed + 1, masked=masked)
        for a, b in zip((w, x, y, lse, dl), new):
            a.copy_(b)
        ws.fill_(0xFF)
        graph.replay()
        assert torch.equal(dx, new[5].float()) and torch.equal(dw, new[6].float()), masked
    assert int(err.item()) == 0


@pytest.mark.parametrize("name", ["lhs_loss", "lhs_loss_grad", "lhs_embed_grad"])
def test_workspace_is_not_handed_out_again(name, monkeypatch):
    # the call's own workspace may be in use on its stream after the call has returned: an
    # allocation of the current stream must not get it
    w, x, y, dl = make(300, 5000, 256, torch.bfloat16)
    tab = table_of(w)
    _, lse, _ = lhs.lhs_loss(tab, x, y)
    ids = torch.arange(300, dtype=torch.int32, device="cuda")
    call = {"lhs_loss": lambda st: lhs.lhs_loss(tab, x, y, stream=st),
            "lhs_loss_grad": lambda st: lhs.lhs_loss_grad(tab, x, y, lse, dl, stream=st),
            "lhs_embed_grad": lambda st: lhs.lhs_embed_grad(ids, x, 5000, 1.0, stream=st)}[name]
    at = {"lhs_loss": 10, "lhs_loss_grad": 16, "lhs_embed_grad": 12}[name]
    real, seen = lhs.lib(), {}

    class Spy:
        def __getattr__(self, fn):
            if fn != name:
                return getattr(real, fn)

            def wrapped(*args):
                seen["ws"] = (args[at], args[at] + args[at + 1])
                return getattr(real, fn)(*args)
            return wrapped

    st = torch.cuda.Stream()
    call(None)
    torch.cuda.synchronize()
    monkeypatch.setattr(lhs, "lib", Spy)
    out = call(st)
    lo, hi = seen["ws"]
    assert hi > lo
    later = [torch.empty(hi - lo, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert all(t.data_ptr() + t.numel() <= lo or t.data_ptr() >= hi for t in later)
    torch.cuda.synchronize()
    del out


def test_tensors_of_wrong_shapes_and_types():
    w, x, y, dl = make(10, 300, 64, torch.bfloat16)
    tab = table_of(w)
    lse = torch.zeros(10, device="cuda")
    half = lhs.lhs_table_init(w.half(), 300, 64, lhs.LHS_F16)
    bad = [lambda: lhs.lhs_loss(tab, x[:, :32], y), lambda: lhs.lhs_loss(half, x, y), lambda: lhs.lhs_loss(tab, x, y[:5]),
           lambda: lhs.lhs_loss(tab, x, y.long()), lambda: lhs.lhs_loss(tab, x.T, y), lambda: lhs.lhs_loss(tab, x, y.cpu()),
           lambda: lhs.lhs_loss(tab, x, y, loss=torch.zeros(9, device="cuda")),
           lambda: lhs.lhs_loss_grad(tab, x, y, lse, dl.double()),
           lambda: lhs.lhs_loss_grad(tab, x, y, lse, dl, accumulate=True),
           lambda: lhs.lhs_loss_grad(tab, x, y, lse, dl, dx=x[:5]),
           lambda: lhs.lhs_loss_grad(tab, x, y, lse, dl, dtable=w[:5]),
           lambda: lhs.lhs_loss_grad(tab, x, y, lse, dl, dtable=w.double()),
           lambda: lhs.lhs_loss_grad(tab, x, y, lse, dl, dtable=torch.zeros((64, 300), device="cuda").T),
           lambda: lhs.lhs_embed_grad(y, x[:5], 300, 1.0), lambda: lhs.lhs_embed_grad(y.long(), x, 300, 1.0),
           lambda: lhs.lhs_embed_grad(y, x, 300, 1.0, accumulate=True),
           lambda: lhs.lhs_embed_grad(y, x, 300, 1.0, dtable=w, dtype=torch.float32),
           lambda: lhs.lhs_embed_grad(y, x, 0, 1.0)]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            assert False, k
    for f in (lambda: lhs.lhs_loss(tab, x, y, temperature=0.0),
              lambda: lhs.lhs_loss(tab, x[:1].expand(10, 64), y),  # rows that overlap
              lambda: lhs.lhs_loss_grad(tab, x, y, lse, dl, want_dx=False, want_dtable=False),
              lambda: lhs.lhs_loss_grad(tab, x, y, lse, dl, dtable=w.half()),
              lambda: lhs.lhs_loss(tab, x, y, ws=torch.empty(256, dtype=torch.uint8, device="cuda")),
              lambda: lhs.lhs_embed_grad(y, x, 300, float("nan"))):
        with pytest.raises(lhs.LhsError):
            f()
