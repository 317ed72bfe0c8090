"""Buffers that overlap are refused by the scoring and training calls, and
buffers that lie side by side, or between the rows of another, are not.
"""
import ctypes

import pytest
import torch

import embedding_lookup_tied_gb300 as lhs
from test_loss import check_grad, check_loss, make, reference, table_of

MB = 1 << 20
T, V, H = 300, 700, 64


def places(*names):
    """Addresses a gigabyte apart (nothing is launched: every call here is refused)."""
    return {n: (k + 1) << 30 for k, n in enumerate(names)}


def c_table(at, vocab=V, hidden=H):
    t = lhs.lhs_table()
    assert lhs.lib().lhs_table_init(ctypes.byref(t), at, vocab, hidden, lhs.LHS_BF16) == 0
    return t


def over(where, a, size, others):
    """`a` moved onto the first and onto the last bytes of each of `others` ({name: bytes}), which it is
    aligned with, and onto its own end."""
    for name, n in others.items():
        for at in (where[name], (where[name] + n - 1) // 256 * 256, where[name] - (size - 1) // 256 * 256):
            if at != where[a]:
                yield name, {**where, a: at}


def test_loss_refuses_overlaps():
    where = places("table", "x", "y", "loss", "lse", "ws", "err")
    L, t = lhs.lib(), c_table(where["table"])
    need = ctypes.c_size_t()
    assert L.lhs_loss_workspace(ctypes.byref(t), T, ctypes.byref(need)) == 0
    size = {"table": V * H * 2, "x": T * H * 2, "y": T * 4, "loss": T * 4, "lse": T * 4, "ws": need.value, "err": 4}
    tried = 0
    for a in ("loss", "lse", "ws", "err"):
        for name, p in over(where, a, size[a], {k: n for k, n in size.items() if k != a}):
            rc = L.lhs_loss(ctypes.byref(t), p["x"], lhs.LHS_BF16, H, T, p["y"], -100, 1.0, p["loss"], p["lse"], p["ws"],
                            need.value, p["err"], None)
            assert rc == lhs.LHS_ERR_INVALID_ARG, (a, name)
            tried += 1
    assert tried == 72


def test_grad_refuses_overlaps():
    where = places("table", "x", "y", "lse", "dl", "dx", "dw", "ws", "err")
    L, t = lhs.lib(), c_table(where["table"])
    need = ctypes.c_size_t()
    assert L.lhs_loss_grad_workspace(ctypes.byref(t), T, ctypes.byref(need)) == 0
    size = {"table": V * H * 2, "x": T * H * 2, "y": T * 4, "lse": T * 4, "dl": T * 4, "dx": T * H * 2, "dw": V * H * 2,
            "ws": need.value, "err": 4}
    for a in ("dx", "dw", "ws", "err"):
        for name, p in over(where, a, size[a], {k: n for k, n in size.items() if k != a and (a, k) != ("dx", "x")}):
            rc = L.lhs_loss_grad(ctypes.byref(t), p["x"], lhs.LHS_BF16, H, T, p["y"], -100, 1.0, p["lse"], p["dl"], p["dx"],
                                 lhs.LHS_BF16, H, p["dw"], lhs.LHS_BF16, 0, p["ws"], need.value, p["err"], None)
            assert rc == lhs.LHS_ERR_INVALID_ARG, (a, name)
    # rows of dx 200 elements apart: one of them lies on the last bytes of the table's gradient
    dx = where["dw"] + size["dw"] - 100 * 400 - 126
    rc = L.lhs_loss_grad(ctypes.byref(t), where["x"], lhs.LHS_BF16, H, T, where["y"], -100, 1.0, where["lse"], where["dl"], dx,
                         lhs.LHS_BF16, 200, where["dw"], lhs.LHS_BF16, 0, where["ws"], need.value, where["err"], None)
    assert rc == lhs.LHS_ERR_INVALID_ARG


@pytest.mark.parametrize("n", [T, 20000])
def test_embed_grad_refuses_overlaps(n):
    where = places("ids", "dout", "dw", "ws", "err")
    L = lhs.lib()
    need = L.lhs_embed_grad_workspace(V, H, n)
    size = {"ids": n * 4, "dout": n * H * 4, "dw": V * H * 4, "ws": need, "err": 4}
    for a in ("dw", "ws", "err"):
        for name, p in over(where, a, size[a], {k: m for k, m in size.items() if k != a}):
            for acc in (0, 1):
                rc = L.lhs_embed_grad(V, H, p["ids"], n, -100, 1.0, p["dout"], lhs.LHS_F32, H, p["dw"], lhs.LHS_F32, acc,
                                      p["ws"], need, p["err"], None)
                assert rc == lhs.LHS_ERR_INVALID_ARG, (a, name)


@pytest.mark.gpu
def test_side_by_side():
    w, x, y, dl = make(T, V, H, torch.bfloat16)
    arena = torch.zeros(64 * MB, dtype=torch.uint8, device="cuda")
    at = 0

    def take(shape, dtype, align=1):
        nonlocal at
        at = (at + align - 1) // align * align
        n = torch.Size(shape).numel() * torch.tensor([], dtype=dtype).element_size()
        t = arena[at:at + n].view(dtype).view(shape)
        at += n
        return t
    # nothing between them but what alignment asks for
    tw = take((V, H), torch.bfloat16)
    tw.copy_(w)
    tab = table_of(tw)
    dw = take((V, H), torch.bfloat16)
    tx = take((T, H), torch.bfloat16)
    tx.copy_(x)
    dx = take((T, H), torch.bfloat16)
    ty, loss, lse, tdl, err = (take((n,), d) for n, d in ((T, torch.int32), (T, torch.float32), (T, torch.float32),
                                                         (T, torch.float32), (1, torch.int32)))
    ty.copy_(y)
    tdl.copy_(dl)
    ws = take((max(lhs.lhs_loss_workspace(tab, T), lhs.lhs_loss_grad_workspace(tab, T)),), torch.uint8, 256)
    lhs.lhs_loss(tab, tx, ty, loss=loss, lse=lse, ws=ws, err=err)
    lhs.lhs_loss_grad(tab, tx, ty, lse, tdl, dx=dx, dtable=dw, ws=ws, err=err)
    r = reference(w, x, y, dl)
    check_loss(loss, lse, r)
    check_grad(dx, dw, r)
    # what is written lies between the rows of what is read
    wide = torch.zeros((T, 2048), dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = x
    gaps = [wide[k, H:H + 2 * T].view(torch.float32) for k in (0, 7)]
    lhs.lhs_loss(tab, wide[:, :H], ty, loss=gaps[0], lse=gaps[1], ws=ws, err=err)
    check_loss(gaps[0], gaps[1], r)
    lhs.lhs_loss_grad(tab, wide[:, :H], ty, lse, tdl, dx=wide[:, 1024:1024 + H], dtable=dw, ws=ws, err=err)
    check_grad(wide[:, 1024:1024 + H], dw, r)
    # one sum's rows beside its gradient
    small = torch.zeros((64, 2 * V * 8), device="cuda")
    rows = small[:, :8]
    rows.copy_(torch.arange(64, device="cuda")[:, None].expand(64, 8))
    ids = torch.arange(64, dtype=torch.int32, device="cuda")
    got, _ = lhs.lhs_embed_grad(ids, rows, V, 1.0, dtable=small[3, 8:8 + 8 * V].view(V, 8), err=err)
    assert torch.equal(got[:64], rows) and bool((got[64:] == 0).all())
    assert int(err.item()) == 0
    for f in (lambda: lhs.lhs_loss(tab, tx, ty, loss=loss, lse=loss), lambda: lhs.lhs_loss_grad(tab, tx, ty, lse, tdl, dx=tx, dtable=tw),
              lambda: lhs.lhs_embed_grad(ids, rows, 64, 1.0, dtable=small.view(-1)[:512].view(64, 8))):
        with pytest.raises(lhs.LhsError):
            f()
