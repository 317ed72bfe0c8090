"""The 8-bit product on its other paths: wide tokens whose rows may be read
several values at a time, rows longer than a warp keeps, rows that are not
finite and captured calls on both kernels, tables of one row; and the
benchmark's cases, small, against their definition.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import embedding_lookup_tied_gb300 as lhs
from test_i8_product import WIDE, make_rows, ref_logits, ref_quantize, same, table_of

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def tokens_of(rng, m, k, dtype, pad=0):
    """Wide tokens [m, k] on rows of k + pad values."""
    return torch.from_numpy(rng.standard_normal((m, k + pad)).astype(np.float32) * 2).to(dtype)


@pytest.mark.parametrize("dtype", WIDE, ids=str)
@pytest.mark.parametrize("m,n,k,pad", [(1, 300, 512, 0), (5, 1000, 896, 0), (12, 257, 132, 0), (40, 300, 512, 0),
                                       (260, 400, 1028, 0), (3, 200, 129, 3), (33, 200, 1001, 3), (7, 200, 130, 6),
                                       (20, 150, 6144, 0), (20, 150, 6148, 0), (20, 150, 9001, 3),
                                       (20, 150, 9001, 0), (18, 100, 13001, 0), (2, 100, 9001, 3)])
def test_aligned_and_long_wide_tokens(dtype, m, n, k, pad):
    rng = np.random.default_rng([m, n, k, pad])
    wb, ws = make_rows(rng, n, k)
    x = tokens_of(rng, m, k, dtype, pad)
    q, s, _ = ref_quantize(x[:, :k].float().numpy())
    out, err = lhs.lhs_i8_logits(table_of(wb, ws, k), x.cuda()[:, :k])
    assert int(err.item()) == 0
    assert same(out, ref_logits(q, s, wb[:, :k], ws, torch.float32))


@pytest.mark.parametrize("dtype", WIDE, ids=str)
@pytest.mark.parametrize("m,k", [(3, 48), (3, 9001), (16, 300), (17, 48), (40, 512), (40, 6500), (260, 130)])
def test_rows_that_are_not_finite(m, k, dtype):
    rng = np.random.default_rng([m, k])
    wb, ws = make_rows(rng, 130, k)
    x = tokens_of(rng, m, k, dtype)
    x[1, 7] = float("inf")
    x[m - 1, k - 1] = float("nan")
    x[0, k // 2] = 0
    out, err = lhs.lhs_i8_logits(table_of(wb, ws, k), x.cuda())
    assert int(err.item()) == lhs.LHS_ERRBIT_NONFINITE
    q, s, bad = ref_quantize(x.float().numpy())
    assert bad and same(out, ref_logits(q, s, wb[:, :k], ws, torch.float32))
    assert bool((out[1] == 0).all()) and bool((out[m - 1] == 0).all()) and bool((out[0] != 0).any())


@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("m", [3, 16, 40, 260])
def test_captured_chain_replays(m, coded):
    # quantise, multiply: three launches of a captured chain, each allowed to start before the last ends
    rng = np.random.default_rng(m)
    n, k = 5000, 896
    w = torch.zeros((n, k), device="cuda")
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    tab, _ = lhs.lhs_i8_quantize(w, err=err)
    tok, _ = lhs.lhs_i8_quantize(x, err=err)
    out = torch.empty((m, n), device="cuda")
    ws = torch.empty(lhs.lhs_i8_workspace(tab, m), dtype=torch.uint8, device="cuda")

    def chain():
        lhs.lhs_i8_quantize(w, codes=tab.tensors[0], scales=tab.tensors[1], err=err)
        if coded:
            lhs.lhs_i8_quantize(x, codes=tok.tensors[0], scales=tok.tensors[1], err=err)
            lhs.lhs_i8_matmul(tok, tab, out=out, ws=ws, err=err)
        else:
            lhs.lhs_i8_logits(tab, x, out=out, ws=ws, err=err)

    chain()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
    for turn in range(3):
        wn = rng.standard_normal((n, k)).astype(np.float32)
        xn = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32)).to(torch.bfloat16)
        w.copy_(torch.from_numpy(wn))
        x.copy_(xn)
        out.fill_(float("nan"))
        g.replay()
        wq, wsc, _ = ref_quantize(wn)
        q, s, _ = ref_quantize(xn.float().numpy())
        assert same(out, ref_logits(q, s, wq, wsc, torch.float32)), turn
    assert int(err.item()) == 0


@pytest.mark.parametrize("m", [2, 30])
@pytest.mark.parametrize("k", [16, 63, 100, 897])
def test_table_of_one_row(m, k):
    # one row of k codes in a buffer that is as wide as a longer table's rows: any number of rows of
    # it is a table, so one is
    rng = np.random.default_rng([m, k])
    wb, ws = make_rows(rng, 5, k)
    ab, as_ = make_rows(rng, m, k)
    codes, scales = torch.from_numpy(wb).cuda(), torch.from_numpy(ws).cuda()
    tok = table_of(ab, as_, k)
    for rows in (2, 1):
        tab = lhs.lhs_i8_init(codes[:rows, :k], scales[:rows], k)
        out, err = lhs.lhs_i8_matmul(tok, tab)
        assert int(err.item()) == 0
        assert same(out, ref_logits(ab[:, :k], as_, wb[:rows, :k], ws[:rows], torch.float32)), rows
    t, _ = lhs.lhs_i8_quantize(torch.from_numpy(wb[:1, :k].astype(np.float32)).cuda())
    again = lhs.lhs_i8_init(t.codes, t.scales, k)
    assert lhs.lhs_i8_matmul(tok, again)[0].shape == (m, 1)


# ---------------------------------------------------------------------------
# the benchmark's cases
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def operators():
    spec = importlib.util.spec_from_file_location("operators", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.own = True
    return m


@pytest.mark.parametrize("m,n,k,x,out", [(1, 700, 96, "f32", "f32"), (9, 515, 100, "bf16", "f16"),
                                         (30, 1001, 333, "f16", "bf16"), (40, 640, 128, "message", "f32"),
                                         (300, 520, 64, "bf16", "bf16")])
def test_benchmark_products(operators, m, n, k, x, out):
    # three binary32 roundings (the sum's and two products') and the output's; where an f16 is subnormal,
    # half of its smallest step
    case = operators.i8_case("small", m, n, k, x, out)
    got = operators.run(operators.prepare(dict(case), 3)).double()
    ref = operators.exact(dict(case), 3).to(got.device)
    dt = operators.DT[out]
    rel = 3 * 2.0 ** -24 + torch.finfo(dt).eps / 2 * (1 + 2.0 ** -20)
    floor = 2.0 ** -25 if dt == torch.float16 else 0.0
    assert got.shape == ref.shape and bool(((got - ref).abs() <= rel * ref.abs() + floor).all())


@pytest.mark.parametrize("b,v,t,mode,masked", [(5, 1000, "f32", "all", False), (12, 3001, "f16", "mixed", True),
                                               (6, 20000, "bf16", "top_p", False), (7, 4096, "f32", "min_p", True),
                                               (4, 5000, "f32", "plain", False), (4, 5000, "f32", "top_k", False)])
def test_benchmark_draws(operators, b, v, t, mode, masked):
    case = operators.sample_case("small", b, v, t, mode, masked)
    got = operators.run(operators.prepare(dict(case), 3))
    ref = operators.exact(dict(case), 3)
    assert got["ids"].cpu().tolist() == ref["ids"].tolist()
    pr = got["probs"].double().cpu().numpy()
    assert (np.abs(pr - ref["probs"]) <= 2.0 ** -23 * ref["probs"]).all()
