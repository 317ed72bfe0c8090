"""Sampling where the weights' accuracy shows: rows so long that a unit of
weight is no longer small.

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

pytestmark = pytest.mark.gpu


def unit_of(v):
    """The unit, in terms of the largest weight (an upper bound)."""
    return 2.0 ** -(min(45, 62 - math.ceil(math.log2(v))) - 1)


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
