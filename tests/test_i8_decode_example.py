"""The decode example, step by step against the definitions: codes, exact
integer logits with their stated roundings, and the draw in 64 bits."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from test_i8_product import ref_logits, ref_quantize
from test_sample import reference

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("i8_decode", os.path.join(ROOT, "examples", "i8_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("vocab,hidden,batch", [(5000, 256, 3), (3001, 100, 20)])
def test_steps_follow_the_definitions(example, vocab, hidden, batch):
    g = torch.Generator().manual_seed(vocab)
    table = torch.randn((vocab, hidden), generator=g).to(torch.bfloat16)
    d = example.Decoder(table.cuda(), batch)
    wq, ws, _ = ref_quantize(table.float().numpy())
    ids = torch.randint(0, vocab, (batch,), generator=g, dtype=torch.int32)
    f = {k: v.cpu() for k, v in d.filters.items()}
    compared = 0
    for _ in range(6):
        u = torch.rand(batch, generator=g)
        nxt, probs = d.step(ids.cuda(), u.cuda())
        xq, xs, _ = ref_quantize(d.x.cpu().numpy())
        ref = ref_logits(xq, xs, wq, ws, torch.float32)
        assert torch.equal(d.logits.cpu(), ref)
        for r in range(batch):
            tok, p, near = reference(ref[r].double().numpy(), float(u[r]), float(f["temperature"][r]),
                                     int(f["top_k"][r]), float(f["top_p"][r]), float(f["min_p"][r]))
            if near:
                continue
            compared += 1
            assert int(nxt[r]) == tok and abs(float(probs[r]) - p) <= 2.0 ** -23 * p
        ids = nxt.cpu().clone()
    assert int(d.err.item()) == 0 and compared >= 5 * batch


def test_main_runs(example):
    t = example.main(["--vocab", "2000", "--hidden", "64", "--batch", "2", "--steps", "5"])
    assert t.shape == (2, 5) and int(t.min()) >= 0 and int(t.max()) < 2000
    again = example.main(["--vocab", "2000", "--hidden", "64", "--batch", "2", "--steps", "5"])
    assert np.array_equal(t.numpy(), again.numpy())
