"""A training step of a tied table as a program runs it: look tokens up, project
the results on the same table, score the next tokens, and add the gradients of
both uses of the table; against the same step in 64 bits.

Tolerances as in test_loss; the lookup's part is exact in f32 up to one rounding
an addition (n 2^-23 of the sum of magnitudes).
"""
import math

import pytest
import torch

import embedding_lookup_tied_gb300 as lhs
from test_loss import CODE, reference, rounding, within

pytestmark = pytest.mark.gpu


class Step:
    """Everything that a step writes is allocated here, once."""

    def __init__(self, table, tokens):
        v, h = table.shape
        dev = table.device
        self.table, self.scale = table, math.sqrt(h)
        self.tab = lhs.lhs_table_init(table, v, h, CODE[table.dtype])
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.rows = torch.empty((tokens, h), device=dev)
        self.x = torch.empty((tokens, h), dtype=table.dtype, device=dev)
        self.loss, self.lse = torch.empty(tokens, device=dev), torch.empty(tokens, device=dev)
        self.dx, self.grad = torch.empty_like(self.x), torch.empty((v, h), device=dev)
        byte = dict(dtype=torch.uint8, device=dev)
        self.ws = torch.empty(max(lhs.lhs_loss_workspace(self.tab, tokens), lhs.lhs_loss_grad_workspace(self.tab, tokens),
                                  lhs.lhs_embed_grad_workspace(v, h, tokens)), **byte)

    def run(self, ids, targets, dloss):
        lhs.lhs_embed(self.tab, ids, self.scale, out=self.rows, err=self.err)
        self.x.copy_(self.rows)  # no model between the two here
        lhs.lhs_loss(self.tab, self.x, targets, loss=self.loss, lse=self.lse, ws=self.ws, err=self.err)
        lhs.lhs_loss_grad(self.tab, self.x, targets, self.lse, dloss, dx=self.dx, dtable=self.grad, ws=self.ws, err=self.err)
        lhs.lhs_embed_grad(ids, self.dx, self.table.shape[0], self.scale, dtable=self.grad, accumulate=True, ws=self.ws,
                           err=self.err)


def batch(t, v, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, v, (t,), generator=g, dtype=torch.int32)
    targets = torch.roll(ids, -1)
    targets[torch.rand(t, generator=g) < 0.2] = -100  # ends of sequences, prompts
    return ids.cuda(), targets.cuda(), (torch.rand(t, generator=g) / t).cuda()


def check(s, ids, targets, dloss):
    r = reference(s.table, s.x, targets, dloss)
    on = r["on"]
    within(s.loss[on], r["loss"], r["tol"])
    within(s.dx[on], r["dx"], r["dx_tol"] + rounding(r["dx"], s.dx.dtype) * 1.01)
    scale = float(torch.tensor(s.scale, dtype=torch.float32))
    own, mag = torch.zeros_like(r["dw"]), torch.zeros_like(r["dw"])
    own.index_add_(0, ids.long(), s.dx.double()).mul_(scale)
    mag.index_add_(0, ids.long(), s.dx.double().abs()).mul_(scale)
    ref = r["dw"] + own
    within(s.grad, ref, r["dw_tol"] + (len(ids) + 2) * 2.0 ** -23 * mag + 2 * rounding(ref, torch.float32) + rounding(r["dw"], torch.float32))
    assert int(s.err.item()) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("t,v,h", [(40, 500, 64), (700, 3000, 136), (300, 40000, 72), (1, 9, 5)])
def test_step(t, v, h, dtype):
    g = torch.Generator().manual_seed(v)
    # a grid, as test_loss has it: the scaled rows' products with the table are exact in f32
    table = (torch.randint(-3, 4, (v, h), generator=g) * 2.0 ** -6).to(dtype).cuda()
    s = Step(table, t)
    s.scale = 4.0
    for seed in range(3):
        b = batch(t, v, seed)
        s.run(*b)
        check(s, *b)


def test_captured_step_while_the_table_changes():
    # an optimiser writes the table between replays; every kernel of the next step reads the new one
    t, v, h = 256, 4000, 128
    g = torch.Generator().manual_seed(3)
    table = (torch.randint(-3, 4, (v, h), generator=g) * 2.0 ** -6).to(torch.bfloat16).cuda()
    s = Step(table, t)
    s.scale = 4.0
    ids, targets, dloss = batch(t, v, 0)
    s.run(ids, targets, dloss)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run(ids, targets, dloss)
    for seed in range(4):
        new = batch(t, v, seed + 1)
        for a, b in zip((ids, targets, dloss), new):
            a.copy_(b)
        table.copy_((torch.randint(-3, 4, (v, h), generator=g) * 2.0 ** -6).to(torch.bfloat16))
        graph.replay()
        check(s, ids, targets, dloss)


def test_gradient_as_a_table_right_after_its_call():
    # the gradient is read as a table (rows looked up, projected) by the calls that follow, which
    # start while the call before is still running
    t, v, h = 600, 30000, 256
    g = torch.Generator().manual_seed(8)
    table = (torch.randn((v, h), generator=g) * 0.05).to(torch.bfloat16).cuda()
    tab = lhs.lhs_table_init(table, v, h, lhs.LHS_BF16)
    x = torch.randn((t, h), generator=g).to(torch.bfloat16).cuda()
    y = torch.randint(0, v, (t,), generator=g, dtype=torch.int32).cuda()
    dl = torch.rand(t, generator=g).cuda()
    _, lse, _ = lhs.lhs_loss(tab, x, y)
    dw = torch.empty_like(table)
    as_table = lhs.lhs_table_init(dw, v, h, lhs.LHS_BF16)
    ids = torch.arange(v - 300, v, dtype=torch.int32, device="cuda")
    few = torch.ones((2, h), device="cuda")
    want = None
    for _ in range(10):
        dw.fill_(float("nan"))
        torch.cuda.synchronize()
        lhs.lhs_loss_grad(tab, x, y, lse, dl, want_dx=False, dtable=dw)
        logits, _ = lhs.lhs_logits(as_table, few)
        dw.fill_(float("nan"))
        lhs.lhs_embed_grad(y, x, v, 2.0, dtable=dw)
        rows, _ = lhs.lhs_embed(as_table, ids, 1.0)
        logits2, _ = lhs.lhs_logits(as_table, few)
        got = [logits, rows, logits2]
        assert all(bool(a.isfinite().all()) for a in got)
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
