"""Sampling where the weights' accuracy shows: unlikely tokens, running sums,
and rows so long that a unit of weight is no longer small.

A row's weights are whole multiples of a unit that is at most 2^-(S-1) of the
largest, S = min(45, 62 - ceil(log2 vocab)), each up to one unit below
its value.  A running sum is therefore up to (its entries) units below its
value, and nowhere above it by more than the weights' own 2^-35.
"""
import math

import numpy as np
import pytest
import torch

import embedding_lookup_tied_gb300 as lhs
from test_sample import reference

pytestmark = pytest.mark.gpu


def unit_of(v):
    """The unit, in terms of the largest weight (an upper bound)."""
    return 2.0 ** -(min(45, 62 - math.ceil(math.log2(v))) - 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("mode", ["none", "k", "p", "q"])
@pytest.mark.parametrize("v", [7, 300, 5000, 300001])
def test_probability_of_unlikely_tokens(v, mode, dtype):
    # u = 0 draws the first id that stays: one that weighs e^-8 .. e^-24 of the largest.  What weighs
    # anything is a few tokens, so the total is good to a few units of 2^-42, and the probability
    # to its own rounding, 2^-24.
    ls = [-8.3, -11.7, -15.1, -18.45, -21.9, -24.3]
    if mode == "p":
        ls = ls[:3]  # weights above the 2^-24 that top-p leaves out
    x = torch.full((len(ls), v), -200.0)
    x[:, v // 2] = 0.4
    x[:, v - 1] = -0.3
    x[:, v - 2] = -30.0
    for r, l in enumerate(ls):
        x[r, 0] = l
    x = x.to(dtype)
    n = len(ls)
    u = torch.zeros(n)
    t = torch.full((n,), 0.97)
    k = torch.full((n,), 3, dtype=torch.int32) if mode == "k" else None
    p = torch.full((n,), 1 - 2.0 ** -24) if mode == "p" else None
    q = torch.full((n,), 2.0 ** -38) if mode == "q" else None
    up = lambda a: None if a is None else a.cuda()  # noqa: E731
    ids, probs, err = lhs.lhs_sample(x.cuda(), u.cuda(), up(t), up(k), up(p), up(q))
    assert int(err.item()) == 0
    for r in range(n):
        tok, pr, near = reference(x[r].double().numpy(), 0.0, float(t[r]), 3 if mode == "k" else 0,
                                  float(p[r]) if p is not None else 1.0, float(q[r]) if q is not None else 0.0)
        assert not near and tok == 0
        assert int(ids[r]) == tok
        assert abs(float(probs[r]) - pr) <= 2.0 ** -23 * pr, (r, float(probs[r]), pr)


@pytest.mark.parametrize("v", [5000, 100003, 262144])
def test_running_sums_are_within_their_units(v):
    # rows of many small weights: the drawn token's stretch of the running sum holds u, up to the
    # units that the sums may be below their values
    g = torch.Generator().manual_seed(v)
    x = torch.randn((3, v), generator=g) * 5
    t = 0.8
    us = torch.cat([torch.rand(60, generator=g), torch.rand(60, generator=g) * 2.0 ** -12,
                    1 - torch.rand(20, generator=g) * 2.0 ** -12]).clamp(max=1 - 2.0 ** -24)
    for r in range(3):
        w = np.exp((x[r].double().numpy() - float(x[r].max())) / float(np.float32(t)))
        c = np.cumsum(w)
        share, slack = c / c[-1], (v + 1) * unit_of(v) / c[-1] + 2.0 ** -35
        n = len(us)
        ids, probs, err = lhs.lhs_sample(x[r].expand(n, v).contiguous().cuda(), us.cuda(),
                                         torch.full((n,), t, device="cuda"))
        assert int(err.item()) == 0
        ids = ids.cpu().numpy()
        uu = us.double().numpy()
        before = np.where(ids > 0, share[np.maximum(ids - 1, 0)], 0.0)
        assert (before <= uu + slack).all() and (uu <= share[ids] + slack).all()
        pr = w[ids] / c[-1]
        assert (np.abs(probs.cpu().numpy() - pr) <= (2.0 ** -23 + slack) * pr).all()


def test_top_p_of_half_a_billion_logits():
    # three large logits and 2^29 - 3 that weigh 1.98 units each: what the units leave out is 4% of
    # the total.  The token has to come from the head that top-p leaves, of the total as it is
    # or less up to one unit an entry, with that head's probability.
    v = 1 << 29
    if torch.cuda.mem_get_info()[0] < 6 << 30:
        pytest.skip("needs 6 GB")
    x = torch.full((1, v), -21.5, dtype=torch.bfloat16, device="cuda")
    at = [12345, v // 2 + 7, v - 3]
    large = torch.tensor([-0.1, 0.0, -0.2]).to(torch.bfloat16)
    for i, l in zip(at, large):
        x[0, i] = l
    w = np.exp(large.double().numpy())
    order = np.argsort(-w)
    head = np.cumsum(w[order])
    small = math.exp(-21.5)
    most = head[-1] + (v - 3) * small
    least = most - (v - 3) * min(small, unit_of(v))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for p in (0.2, 0.348, 0.35, 0.5, 0.666, 0.667, 0.668, 0.8):
        p32 = float(np.float32(p))
        sizes = {int(np.searchsorted(head, p32 * total, side="left")) + 1 for total in (least, most)}
        assert max(sizes) <= 3
        for u in (0.0, 0.3, 0.6, 0.97):
            ids, probs, _ = lhs.lhs_sample(x, torch.tensor([u]).cuda(), top_p=torch.tensor([p]).cuda(),
                                           ids=torch.full((1,), -7, dtype=torch.int32, device="cuda"),
                                           probs=torch.full((1,), -7.0, device="cuda"), err=err)
            right = []
            for n in sizes:
                keep = np.sort(order[:n])  # the large ones' ids ascend with their numbers here
                c = np.cumsum(w[keep])
                k = keep[int(np.searchsorted(c, float(np.float32(u)) * c[-1], side="right"))]
                right.append((at[k], w[k] / c[-1]))
            got = (int(ids.item()), float(probs.item()))
            # of three weights at most, a few units of 2^-32 off: within the rounding's 2^-23
            assert any(got[0] == i and abs(got[1] - q) <= 2.0 ** -23 * q for i, q in right), (p, u, got, right)
    assert int(err.item()) == 0
