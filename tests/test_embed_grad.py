"""The gradient of the scaled lookup, against sums in 64 bits.

Where the rows hold small integers every sum is exact in f32, whatever its
order: the result is then the exact product with the scale, rounded to f32 and
to the output's type, and compared for equality.  Random rows: m positions of
an id are m additions of 2^-24 each, of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import embedding_lookup_tied_gb300 as lhs

FAKE = 0x10000
WIDE = [torch.float32, torch.float16, torch.bfloat16]


def test_refuses():
    L = lhs.lib()
    big = 1 << 40

    def call(v=100, h=16, ids=FAKE, n=5, scale=1.0, d=FAKE, dt=0, ds=16, o=FAKE, ot=0, acc=0, ws=FAKE, wb=big, err=FAKE):
        return L.lhs_embed_grad(v, h, ids, n, -100, scale, d, dt, ds, o, ot, acc, ws, wb, err, None)
    for bad in (dict(v=0), dict(v=2 ** 31), dict(h=0), dict(h=65537, ds=65537), dict(n=-1), dict(n=2 ** 30 + 1), dict(ids=None),
                dict(ids=FAKE + 2), dict(scale=float("nan")), dict(scale=float("inf")), dict(d=None), dict(d=FAKE + 2),
                dict(d=FAKE + 1, dt=1), dict(dt=3), dict(dt=-1), dict(ds=15), dict(o=None), dict(o=FAKE + 8),
                dict(ot=3), dict(ot=4), dict(acc=2), dict(ws=None), dict(ws=FAKE + 64), dict(err=None),
                dict(err=FAKE + 2)):
        assert call(**bad) == lhs.LHS_ERR_INVALID_ARG, bad
    need = L.lhs_embed_grad_workspace(100, 16, 5)
    assert need > 0 and call(wb=need - 1) == lhs.LHS_ERR_BUFFER_TOO_SMALL
    assert call(n=0, acc=1, ids=None, d=None, ws=None, wb=0, err=None) == lhs.LHS_OK
    for v, h, n in ((0, 16, 5), (100, 0, 5), (100, 16, -1), (2 ** 31, 16, 5), (100, 65537, 5), (100, 16, 2 ** 30 + 1)):
        assert L.lhs_embed_grad_workspace(v, h, n) == -1


def test_binding_refuses_cpu_tensors():
    with pytest.raises(ValueError):
        lhs.lhs_embed_grad(torch.zeros(2, dtype=torch.int32), torch.zeros((2, 8)), 10, 1.0)


def zipf(n, v, g):
    c = torch.cumsum(torch.arange(1, v + 1, dtype=torch.float64) ** -1.1, 0)
    r = torch.searchsorted(c, torch.rand(n, generator=g, dtype=torch.float64) * c[-1]).clamp(max=v - 1)
    return torch.randperm(v, generator=g)[r].to(torch.int32)


def sums(ids, rows, v, ignore=-100):
    ok = (ids >= 0) & (ids < v) & (ids != ignore)
    out = torch.zeros((v, rows.shape[1]), dtype=torch.float64, device=rows.device)
    return out.index_add_(0, ids[ok].long(), rows[ok].double())


SIZES = [(1, 1, 1), (1, 100, 8), (2, 3, 5), (5, 7, 33), (16, 8192, 256), (31, 50, 100), (100, 1, 64), (333, 1000, 1001),
         (1000, 40, 24), (628, 15000, 896), (2048, 5000, 64), (4097, 300, 130), (8192, 30000, 40), (8193, 2000, 36),
         (20000, 70000, 16), (40000, 3, 8), (70001, 9000, 12), (100000, 300000, 4), (300001, 20000, 24), (600000, 500, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,v,h", SIZES)
@pytest.mark.parametrize("dtype", WIDE, ids=str)
def test_sizes(n, v, h, dtype):
    g = torch.Generator().manual_seed(n + v * 3 + h)
    ids = zipf(n, v, g).cuda()
    rows = torch.randint(-8, 9, (n, h), generator=g).to(dtype).cuda()
    scale = float(np.float32(h ** 0.5))
    ref = sums(ids, rows, v) * scale
    for out in WIDE:
        d, err = lhs.lhs_embed_grad(ids, rows, v, scale, dtype=out)
        assert int(err.item()) == 0
        assert torch.equal(d, ref.float().to(out)), out
    base = torch.randint(-50, 51, (v, h), generator=g).to(dtype).cuda()
    d = base.clone()
    lhs.lhs_embed_grad(ids, rows, v, 0.5, dtable=d, accumulate=True)
    assert torch.equal(d, (base.double() + 0.5 * sums(ids, rows, v)).float().to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("n,v,h", [(700, 50, 100), (9000, 4000, 72), (60000, 100, 20)])
@pytest.mark.parametrize("dtype", WIDE, ids=str)
def test_random_rows(n, v, h, dtype):
    g = torch.Generator().manual_seed(n)
    ids = zipf(n, v, g).cuda()
    rows = (torch.randn((n, h), generator=g) * torch.rand((n, 1), generator=g)).to(dtype).cuda()
    ref, mag = sums(ids, rows, v) * 3.0, sums(ids, rows.abs(), v) * 3.0
    m = torch.bincount(ids.long(), minlength=v)[:, None].double()
    for out in WIDE:
        d, _ = lhs.lhs_embed_grad(ids, rows, v, 3.0, dtype=out)
        tol = (m + 1) * 2.0 ** -24 * mag + torch.finfo(out).eps / 2 * ref.abs() * 1.01 + (2.0 ** -25 if out == torch.float16 else 0)
        assert bool(((d.double() - ref).abs() <= tol).all())
        again, _ = lhs.lhs_embed_grad(ids, rows, v, 3.0, dtype=out)
        assert torch.equal(d, again)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 9, 500, 9000, 30000])
def test_ids_that_take_no_part(n):
    g = torch.Generator().manual_seed(n)
    v, h = 60, 40
    ids = torch.randint(0, v, (n,), generator=g, dtype=torch.int32)
    ids[torch.rand(n, generator=g) < 0.4] = -100
    bad = n > 8
    if bad:
        ids[2:6] = torch.tensor([-1, v, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    rows = torch.randint(-8, 9, (n, h), generator=g).float()
    rows[(ids < 0) | (ids >= v)] = float("nan")  # reaches nothing
    ids, rows = ids.cuda(), rows.cuda()
    d, err = lhs.lhs_embed_grad(ids, rows, v, 1.0)
    assert int(err.item()) == (lhs.LHS_ERRBIT_BAD_TOKEN if bad else 0)
    assert torch.equal(d, sums(ids, rows, v).float())
    ids.fill_(7)  # an id to ignore inside the vocabulary; nothing is left
    d, err = lhs.lhs_embed_grad(ids, rows, v, 1.0, ignore=7)
    assert int(err.item()) == 0 and bool((d == 0).all())
    d.fill_(5.0)
    lhs.lhs_embed_grad(ids, rows, v, 1.0, dtable=d, accumulate=True, ignore=7)
    assert bool((d == 5).all())


@pytest.mark.gpu
@pytest.mark.parametrize("h", [16, 33, 256])
@pytest.mark.parametrize("dtype", WIDE, ids=str)
def test_strides_and_addresses(h, dtype):
    g = torch.Generator().manual_seed(h)
    n, v = 3000, 500
    ids = zipf(n, v, g).cuda()
    wide = torch.full((n, h + 11), float("nan"), dtype=dtype, device="cuda")
    for off in (0, 1, 8):
        rows = wide[:, off:off + h]
        rows.copy_(torch.randint(-8, 9, (n, h), generator=g))
        d, err = lhs.lhs_embed_grad(ids, rows, v, 2.0, dtype=dtype)
        assert int(err.item()) == 0 and torch.equal(d, (2 * sums(ids, rows, v)).float().to(dtype))
        rows.fill_(float("nan"))


@pytest.mark.gpu
def test_same_id_everywhere_and_each_once():
    g = torch.Generator().manual_seed(4)
    for n, v, h in ((50000, 10, 24), (8192, 8192, 16), (30000, 30000, 16)):
        rows = torch.randint(-4, 5, (n, h), generator=g).to(torch.bfloat16).cuda()
        one = torch.full((n,), v - 1, dtype=torch.int32, device="cuda")
        d, _ = lhs.lhs_embed_grad(one, rows, v, 1.0)
        assert torch.equal(d, sums(one, rows, v).float())
        each = torch.randperm(n, generator=g).remainder(v).to(torch.int32).cuda()
        d, _ = lhs.lhs_embed_grad(each, rows, v, 1.0)
        assert torch.equal(d, sums(each, rows, v).float())


@pytest.mark.gpu
def test_values_that_are_not_finite():
    ids = torch.tensor([3, 1, 3, 2, 1], dtype=torch.int32, device="cuda")
    rows = torch.ones((5, 8), device="cuda")
    rows[0, 0], rows[2, 0], rows[1, 1] = float("inf"), float("-inf"), float("nan")
    rows[3, 2] = 3e38
    d, err = lhs.lhs_embed_grad(ids, rows, 5, 2.0)
    assert int(err.item()) == 0
    assert bool(d[3, 0].isnan()) and bool(d[1, 1].isnan()) and bool(d[2, 2] == float("inf"))
    d[3, 0] = d[1, 1] = d[2, 2] = 0
    ref = 2 * sums(ids, torch.ones_like(rows), 5).float()
    ref[3, 0] = ref[1, 1] = ref[2, 2] = 0
    assert torch.equal(d, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [500, 20000])
def test_captured_call_replays(n):
    v, h = 4000, 64
    g = torch.Generator().manual_seed(n)
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    rows = torch.zeros((n, h), device="cuda")
    d = torch.empty((v, h), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(lhs.lhs_embed_grad_workspace(v, h, n), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lhs.lhs_embed_grad(ids, rows, v, 1.0, dtable=d, ws=ws, err=err)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lhs.lhs_embed_grad(ids, rows, v, 1.0, dtable=d, ws=ws, err=err)
    for _ in range(3):
        ids.copy_(zipf(n, v, g))
        rows.copy_(torch.randint(-8, 9, (n, h), generator=g))
        ws.fill_(0xFF)
        graph.replay()
        assert torch.equal(d, sums(ids, rows, v).float().to(torch.bfloat16))
    assert int(err.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n", [700, 30000])
def test_streams(n):
    v, h = 3000, 128
    g = torch.Generator().manual_seed(n)
    data = [(zipf(n, v, g).cuda(), torch.randint(-8, 9, (n, h), generator=g).float().cuda()) for _ in range(2)]
    refs = [sums(i, r, v).float() for i, r in data]
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        torch.cuda._sleep(5_000_000)
        got = [lhs.lhs_embed_grad(i, r, v, 1.0, stream=s) for (i, r), s in zip(data, st)]
        torch.cuda.synchronize()
        for (d, err), ref in zip(got, refs):
            assert torch.equal(d, ref) and int(err.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,h", [(300, 33), (9000, 16)])
def test_nothing_else_is_written(n, h):
    from gpu_util import canaries_intact, guarded
    v = 501
    g = torch.Generator().manual_seed(n)
    ids, rows = zipf(n, v, g).cuda(), torch.randint(-8, 9, (n, h), generator=g).to(torch.float16).cuda()
    raw, d, pad = guarded((v, h), torch.float16)
    raww, ws, padw = guarded((lhs.lhs_embed_grad_workspace(v, h, n),), torch.uint8)
    lhs.lhs_embed_grad(ids, rows, v, 1.0, dtable=d, ws=ws)
    assert torch.equal(d, sums(ids, rows, v).float().to(torch.float16))
    assert canaries_intact(raw, pad) and canaries_intact(raww, padw)


@pytest.mark.gpu
def test_offsets_pass_32_bits():
    v, h, n = 1_500_000, 2048, 1_100_000
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    ids = torch.arange(n, dtype=torch.int32, device="cuda") + (v - n)
    ids[0] = v - 1
    rows = torch.zeros((n, h), dtype=torch.bfloat16, device="cuda")
    rows[-1] = 3.0
    rows[0] = 4.0
    rows[-2, 5] = 2.0
    d, err = lhs.lhs_embed_grad(ids, rows, v, 1.0, dtype=torch.bfloat16)
    assert int(err.item()) == 0
    assert bool((d[-1] == 7).all()) and float(d[-2, 5]) == 2.0 and float(d[-2].float().sum()) == 2.0
    assert float(d[:-2].abs().max()) == 0.0


@pytest.mark.gpu
def test_ids_of_29_bits():
    # four passes over the digits
    v, n = (1 << 28) + 5, 9000
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    g = torch.Generator().manual_seed(2)
    ids = torch.randint(0, v, (n,), generator=g, dtype=torch.int32)
    ids[:4000] = ids[4000:8000]
    ids[:3] = torch.tensor([v - 1, 0, v - 1], dtype=torch.int32)
    rows = torch.randint(-8, 9, (n, 1), generator=g).to(torch.bfloat16)
    d, err = lhs.lhs_embed_grad(ids.cuda(), rows.cuda(), v, 1.0, dtype=torch.bfloat16)
    at, inv = torch.unique(ids.long(), return_inverse=True)
    ref = torch.zeros(len(at), dtype=torch.float64).index_add_(0, inv, rows[:, 0].double())
    assert int(err.item()) == 0 and torch.equal(d[at.cuda(), 0].cpu(), ref.to(torch.bfloat16))
    d[at.cuda()] = 0
    assert int(torch.count_nonzero(d)) == 0


@pytest.mark.gpu
def test_is_the_transpose_of_the_lookup():
    # <lookup(T), G> = <T, gradient(G)> for any T and G
    g = torch.Generator().manual_seed(9)
    v, h, n = 700, 64, 3000
    table = torch.randint(-3, 4, (v, h), generator=g).float().cuda()
    ids = zipf(n, v, g).cuda()
    rows = torch.randint(-3, 4, (n, h), generator=g).float().cuda()
    out, _ = lhs.lhs_embed(lhs.lhs_table_init(table, v, h, lhs.LHS_F32), ids, 4.0)
    d, _ = lhs.lhs_embed_grad(ids, rows, v, 4.0)
    assert float((out.double() * rows.double()).sum()) == float((table.double() * d.double()).sum())
