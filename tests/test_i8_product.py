"""Rows in 8 bits: quantisation, the product of tokens and channels in int8
with one scale each, and the refusals of both.

The sums of codes are integers and the roundings after them are stated, so the
expected logits are formed in int64 and in single binary32 operations, and
the comparison is for equal values, with no tolerance.
"""
import ctypes

import numpy as np
import pytest
import torch

import embedding_lookup_tied_gb300 as lhs
import oracle as orc
from gpu_util import canaries_intact, guarded

FAKE = 0x10000  # an aligned address that these calls never dereference
WIDE = [torch.float32, torch.float16, torch.bfloat16]


# ---------------------------------------------------------------------------
# refusals (CPU)
# ---------------------------------------------------------------------------
def _desc(codes=FAKE, stride=64, scales=FAKE, sstride=4, rows=10, hidden=64):
    t = lhs.lhs_i8()
    rc = lhs.lib().lhs_i8_init(ctypes.byref(t), codes, stride, scales, sstride, rows, hidden)
    return rc, t


def test_init_refuses():
    assert _desc()[0] == lhs.LHS_OK
    assert _desc(rows=0, codes=None, scales=None)[0] == lhs.LHS_OK
    for bad in (dict(codes=None), dict(scales=None), dict(scales=FAKE + 2), dict(rows=-1), dict(rows=2 ** 31),
                dict(hidden=0), dict(hidden=65), dict(hidden=(1 << 24) + 1, stride=1 << 25), dict(sstride=2),
                dict(sstride=6), dict(sstride=0), dict(stride=-64)):
        assert _desc(**bad)[0] == lhs.LHS_ERR_INVALID_ARG, bad
    assert lhs.lib().lhs_i8_init(None, FAKE, 64, FAKE, 4, 10, 64) == lhs.LHS_ERR_INVALID_ARG


def test_message_refuses():
    L, t = lhs.lib(), lhs.lhs_i8()
    need = L.lhs_wire_bytes(lhs.LHS_WIRE_I8, 3, 64)
    assert L.lhs_i8_message(ctypes.byref(t), FAKE, need, 16, 3, 64) == lhs.LHS_OK
    assert (t.codes, t.scales, t.rows, t.stride, t.scale_stride, t.hidden, t.header) == \
        (FAKE + 24, FAKE + 16, 3, 72, 72, 64, 16)
    assert L.lhs_i8_message(ctypes.byref(t), FAKE + 4, need - 4, 12, 3, 64) == lhs.LHS_OK
    assert t.codes == FAKE + 4 + 20
    assert L.lhs_i8_message(ctypes.byref(t), FAKE, need - 1, 16, 3, 64) == lhs.LHS_ERR_BUFFER_TOO_SMALL
    for args in ((None, need, 16, 3, 64), (FAKE + 2, need, 16, 3, 64), (FAKE, need, 8, 3, 64),
                 (FAKE, need, 16, -1, 64), (FAKE, need, 16, 3, 66), (FAKE, need, 16, 3, 0)):
        assert L.lhs_i8_message(ctypes.byref(t), *args) == lhs.LHS_ERR_INVALID_ARG, args


def test_quantize_refuses():
    L = lhs.lib()
    _, t = _desc()
    q = lambda t=t, x=FAKE, dt=0, xs=64, err=FAKE: L.lhs_i8_quantize(ctypes.byref(t), x, dt, xs, err, None)  # noqa: E731
    for bad in (dict(x=None), dict(x=FAKE + 2), dict(dt=lhs.LHS_Q8_0), dict(dt=9), dict(xs=63), dict(err=None),
                dict(err=FAKE + 1), dict(x=FAKE + 1, dt=lhs.LHS_F16)):
        assert q(**bad) == lhs.LHS_ERR_INVALID_ARG, bad
    assert q(t=_desc(rows=0)[1], x=None, err=None) == lhs.LHS_OK  # nothing to do
    m = lhs.lhs_i8()
    L.lhs_i8_message(ctypes.byref(m), FAKE, 1 << 20, 16, 3, 64)
    assert q(t=m) == lhs.LHS_ERR_INVALID_ARG


def test_product_refuses():
    L = lhs.lib()
    _, w = _desc(rows=100)
    _, a = _desc(rows=5)
    n = ctypes.c_size_t()
    assert L.lhs_i8_workspace(ctypes.byref(w), 5, ctypes.byref(n)) == lhs.LHS_OK and n.value > 0
    assert L.lhs_i8_workspace(ctypes.byref(w), -1, ctypes.byref(n)) == lhs.LHS_ERR_INVALID_ARG
    assert L.lhs_i8_workspace(ctypes.byref(w), 5, None) == lhs.LHS_ERR_INVALID_ARG

    def mm(w=w, a=a, out=FAKE, dt=0, os=100, ws=FAKE, nb=n.value, err=FAKE):
        return L.lhs_i8_matmul(ctypes.byref(a), ctypes.byref(w), out, dt, os, ws, nb, err, None)

    def lg(w=w, x=FAKE, xdt=0, xs=64, t=5, out=FAKE, dt=0, os=100, ws=FAKE, nb=n.value, err=FAKE):
        return L.lhs_i8_logits(ctypes.byref(w), x, xdt, xs, t, out, dt, os, ws, nb, err, None)

    for bad in (dict(out=None), dict(out=FAKE + 2), dict(dt=lhs.LHS_Q8_0), dict(os=99), dict(ws=None),
                dict(ws=FAKE + 16), dict(err=None), dict(err=FAKE + 2),
                dict(w=_desc(codes=FAKE + 8)[1]), dict(w=_desc(stride=72)[1])):
        assert mm(**bad) == lhs.LHS_ERR_INVALID_ARG, bad
        assert lg(**bad) == lhs.LHS_ERR_INVALID_ARG, bad
    for bad in (dict(x=None), dict(x=FAKE + 2), dict(xdt=lhs.LHS_FP8_E4M3), dict(xs=63), dict(t=-1)):
        assert lg(**bad) == lhs.LHS_ERR_INVALID_ARG, bad
    assert mm(a=_desc(hidden=63)[1]) == lhs.LHS_ERR_INVALID_ARG
    assert mm(w=_desc(hidden=131072, stride=131072)[1], a=_desc(hidden=131072, stride=131072)[1]) == \
        lhs.LHS_ERR_INVALID_ARG  # a sum could pass 2^31
    assert mm(nb=n.value - 1) == lhs.LHS_ERR_BUFFER_TOO_SMALL
    assert lg(nb=n.value - 1) == lhs.LHS_ERR_BUFFER_TOO_SMALL
    assert mm(a=_desc(rows=0)[1], out=None, ws=None) == lhs.LHS_OK
    assert mm(w=_desc(rows=0)[1], os=0, out=None, ws=None) == lhs.LHS_OK
    m = lhs.lhs_i8()
    L.lhs_i8_message(ctypes.byref(m), FAKE, 1 << 20, 16, 3, 64)
    assert mm(w=m) == lhs.LHS_ERR_INVALID_ARG  # a table is plain rows


def test_binding_refuses_cpu_tensors():
    with pytest.raises(ValueError):
        lhs.lhs_i8_init(torch.zeros((2, 16), dtype=torch.int8), torch.zeros(2), 16)
    with pytest.raises(ValueError):
        lhs.lhs_i8_quantize(torch.zeros((2, 16)))


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------
def ref_quantize(x):
    """(codes, scales, whether any row is not finite) by the definition, in
    single binary32 operations."""
    x = x.astype(np.float32)
    bad = ~np.isfinite(x).all(1)
    top = np.abs(np.where(bad[:, None], 0, x)).max(1).astype(np.float32)
    scale = top / np.float32(127)
    with np.errstate(over="ignore", invalid="ignore"):
        q = np.where(bad[:, None], 0, x) / np.where(scale > 0, scale, np.float32(1))[:, None]
    q = np.where(scale[:, None] > 0, np.clip(np.rint(q), -127, 127), 0)
    return q.astype(np.int8), scale, bool(bad.any())


def ref_logits(a, a_scale, w, w_scale, dtype):
    """The definition: int64 sums, then one binary32 rounding per step."""
    acc = (torch.from_numpy(a).double() @ torch.from_numpy(w).double().T).numpy()  # exact: below 2^53
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        v = acc.astype(np.float32) * a_scale[:, None].astype(np.float32) * w_scale[None, :].astype(np.float32)
    return torch.from_numpy(v).to(dtype)


def same(got, ref):
    got, ref = got.cpu().float(), ref.float()
    return got.shape == ref.shape and bool(((got == ref) | (got.isnan() & ref.isnan())).all())


def make_rows(rng, rows, hidden, pad=0, lowest=-127):
    """Codes on rows of a 16-byte multiple (pad more of them), junk between."""
    stride = (hidden + 15) // 16 * 16 + 16 * pad
    buf = rng.integers(-128, 128, (rows, stride), dtype=np.int8)
    buf[:, :hidden] = rng.integers(lowest, 128, (rows, hidden), dtype=np.int8)
    return buf, rng.uniform(1e-4, 2e-2, rows).astype(np.float32)


def table_of(buf, scales, hidden):
    return lhs.lhs_i8_init(torch.from_numpy(buf).cuda(), torch.from_numpy(scales).cuda(), hidden)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", WIDE, ids=str)
@pytest.mark.parametrize("rows,hidden", [(1, 1), (3, 2), (5, 17), (300, 31), (7, 128), (33, 896), (4, 1001),
                                         (2, 1024), (2, 1030), (9, 5376), (3, 8192), (2, 20003), (1100, 64), (0, 16)])
def test_quantize(dtype, rows, hidden):
    g = torch.Generator().manual_seed(rows * 7 + hidden)
    x = torch.randn((rows, hidden + 3), generator=g) * 3
    x = x.to(dtype)
    if rows > 3:
        x[1] = 0  # an all-zero row
        x[3, :hidden] = x[3, :hidden].abs().max()  # every code 127
    xd = x.cuda()[:, 1:hidden + 1]  # rows that start off any wider alignment
    stride = (hidden + 15) // 16 * 16 + 16
    raw, codes, pad = guarded((rows, stride), torch.int8)
    t, err = lhs.lhs_i8_quantize(xd, codes=codes)
    q, s, _ = ref_quantize(x[:, 1:hidden + 1].float().numpy()) if rows else (np.zeros((0, hidden), np.int8),
                                                                              np.zeros(0, np.float32), False)
    assert int(err.item()) == 0
    assert np.array_equal(t.scales.cpu().numpy(), s)
    assert np.array_equal(t.codes.cpu().numpy(), q)
    assert canaries_intact(raw, pad)
    assert bool((codes[:, hidden:] == 0x5A).all())  # the gap between rows is not written
    if rows:  # codes and values at any address
        odd = torch.full((rows, hidden + 6), 90, dtype=torch.int8, device="cuda")
        t, _ = lhs.lhs_i8_quantize(xd.contiguous(), codes=odd[:, 3:hidden + 3])
        assert np.array_equal(t.codes.cpu().numpy(), q) and np.array_equal(t.scales.cpu().numpy(), s)
        assert bool((odd[:, :3] == 90).all()) and bool((odd[:, hidden + 3:] == 90).all())


@pytest.mark.gpu
def test_quantize_special_values():
    h = 70
    x = np.random.default_rng(3).standard_normal((9, h)).astype(np.float32)
    x[0, 5] = np.inf
    x[1, 69] = np.nan
    x[2] = 0
    x[3] = 1e-44  # a subnormal scale: max / 127 rounds to 0
    x[4] *= 1e-37
    x[5] *= np.float32(3e38) / np.abs(x[5]).max()
    x[6] = np.float32(63.5) * np.sign(x[6])  # quotients at +-127
    x[7] = np.arange(h) + 0.5
    x[7, 0] = 127.0  # scale 1: every code a tie
    t, err = lhs.lhs_i8_quantize(torch.from_numpy(x).cuda())
    q, s, bad = ref_quantize(x)
    assert bad and int(err.item()) == lhs.LHS_ERRBIT_NONFINITE
    assert np.array_equal(t.scales.cpu().numpy(), s) and np.array_equal(t.codes.cpu().numpy(), q)


SIZES = [(1, 1, 1), (1, 128, 64), (1, 129, 65), (2, 127, 16), (1, 1000, 896), (3, 257, 15), (8, 300, 17), (4, 5000, 300), (5, 40001, 130), (11, 21000, 256),
         (9, 640, 63), (16, 255, 127), (17, 513, 128), (31, 100, 129), (33, 1001, 1001), (64, 320, 768),
         (65, 130, 192), (128, 256, 1024), (129, 383, 1025), (200, 70, 333), (256, 512, 2048), (257, 200, 2100),
         (300, 129, 64), (513, 777, 100), (640, 2000, 320)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", SIZES)
def test_matmul_sizes(m, n, k):
    rng = np.random.default_rng([m, n, k])
    wb, ws = make_rows(rng, n, k, pad=n % 2)
    ab, as_ = make_rows(rng, m, k)
    tab, tok = table_of(wb, ws, k), table_of(ab, as_, k)
    for dtype in WIDE:
        raw, out, pad = guarded((m, n), dtype)
        _, err = lhs.lhs_i8_matmul(tok, tab, out=out)
        assert int(err.item()) == 0
        assert same(out, ref_logits(ab[:, :k], as_, wb[:, :k], ws, dtype)), dtype
        assert canaries_intact(raw, pad)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 2, 3, 7, 14, 20, 140, 260])
@pytest.mark.parametrize("k", [1023, 1024, 1025, 2047, 3000, 9000, 40000, 131071])
def test_matmul_sums_are_exact(m, k):
    # codes at the ends of the range with few signs: sums far beyond 2^24, up to 2^31
    rng = np.random.default_rng([m, k])
    n = 150
    wb, ws = make_rows(rng, n, k)
    ab, as_ = make_rows(rng, m, k)
    wb[:, :k] = np.where(rng.random((n, k)) < 0.01, 126, -128)
    ab[:, :k] = np.where(rng.random((m, k)) < 0.01, 127, -128)
    wb[:5, :k] = -128
    ab[0, :k] = -128
    ws[:], as_[:] = 1.0, 1.0
    out, err = lhs.lhs_i8_matmul(table_of(ab, as_, k), table_of(wb, ws, k))
    assert int(err.item()) == 0
    assert same(out, ref_logits(ab[:, :k], as_, wb[:, :k], ws, torch.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", WIDE, ids=str)
@pytest.mark.parametrize("m,n,k", [(1, 1000, 896), (1, 77, 33), (5, 300, 1001), (40, 129, 130), (150, 260, 64)])
def test_logits_is_quantize_then_matmul(dtype, m, n, k):
    rng = np.random.default_rng([m, n, k, 1])
    wb, ws = make_rows(rng, n, k)
    x = torch.from_numpy(rng.standard_normal((m, k + 5)).astype(np.float32)).to(dtype)
    xd = x.cuda()[:, 2:k + 2]
    q, s, _ = ref_quantize(x[:, 2:k + 2].float().numpy())
    tab = table_of(wb, ws, k)
    for od in WIDE:
        out, err = lhs.lhs_i8_logits(tab, xd, out_dtype=od)
        assert int(err.item()) == 0
        assert same(out, ref_logits(q, s, wb[:, :k], ws, od))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 24, 200])
def test_strided_outputs_and_tokens(m):
    rng = np.random.default_rng(m)
    n, k = 211, 150
    wb, ws = make_rows(rng, n, k, pad=3)
    ab = rng.integers(-127, 128, (m, 157), dtype=np.int8)  # token rows at odd addresses
    as_ = rng.uniform(0.1, 1, (m, 3)).astype(np.float32)
    tok = lhs.lhs_i8_init(torch.from_numpy(ab).cuda()[:, 3:], torch.from_numpy(as_).cuda()[:, 1], k)
    wsd = torch.from_numpy(np.repeat(ws, 2)).cuda()[::2]  # scales two apart
    tab = lhs.lhs_i8_init(torch.from_numpy(wb).cuda(), wsd, k)
    for dtype in WIDE:
        big = torch.full((m, n + 14), 7.0, dtype=dtype, device="cuda")
        out = big[:, 5:5 + n]
        lhs.lhs_i8_matmul(tok, tab, out=out)
        assert same(out, ref_logits(ab[:, 3:3 + k], as_[:, 1], wb[:, :k], ws, dtype))
        assert bool((big[:, :5] == 7).all()) and bool((big[:, 5 + n:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("m", [2, 70])
def test_special_scales(m):
    rng = np.random.default_rng(9)
    n, k = 140, 96
    wb, ws = make_rows(rng, n, k)
    ab, as_ = make_rows(rng, m, k)
    ws[:6] = [0, np.inf, np.nan, 1e38, 1e-45, -0.5]
    as_[:2] = [0, 1e30]
    wb[7, :k] = 0
    out, _ = lhs.lhs_i8_matmul(table_of(ab, as_, k), table_of(wb, ws, k))
    assert same(out, ref_logits(ab[:, :k], as_, wb[:, :k], ws, torch.float32))
    for dtype in (torch.float16, torch.bfloat16):  # beyond the f16 range: inf
        out, _ = lhs.lhs_i8_matmul(table_of(ab, as_, k), table_of(wb, ws, k), out_dtype=dtype)
        assert same(out, ref_logits(ab[:, :k], as_, wb[:, :k], ws, dtype))


@pytest.mark.gpu
def test_nonfinite_tokens():
    rng = np.random.default_rng(4)
    wb, ws = make_rows(rng, 130, 48)
    x = rng.standard_normal((3, 48)).astype(np.float32)
    x[1, 7] = np.inf
    out, err = lhs.lhs_i8_logits(table_of(wb, ws, 48), torch.from_numpy(x).cuda())
    assert int(err.item()) == lhs.LHS_ERRBIT_NONFINITE
    q, s, _ = ref_quantize(x)
    assert same(out, ref_logits(q, s, wb[:, :48], ws, torch.float32)) and bool((out[1] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("response", [False, True])
@pytest.mark.parametrize("m,k", [(1, 896), (9, 132), (64, 768), (130, 100)])
def test_message_tokens(response, m, k):
    rng = np.random.default_rng([m, k, response])
    wb, ws = make_rows(rng, 300, k)
    tab = table_of(wb, ws, k)
    x = rng.standard_normal((m, k)).astype(np.float32)
    xd = torch.from_numpy(x).cuda()
    enc = lhs.lhs_wire_encode_response if response else lhs.lhs_wire_encode
    buf, _ = enc(lhs.LHS_WIRE_I8, xd)
    out, err = lhs.lhs_i8_matmul(lhs.lhs_i8_message(buf, m, k, response), tab)
    q, s, _ = ref_quantize(x)
    assert int(err.item()) == 0
    ref = ref_logits(q, s, wb[:, :k], ws, torch.float32)
    assert same(out, ref)
    # a position with a zero point: that token's results are NaN
    head = 12 if response else 16
    bad = buf.clone() if not response else torch.cat([buf.new_zeros(4), buf])[4:]
    p = head + (m - 1) * (k + 8) + 4
    bad[p:p + 4] = torch.tensor([1.0]).view(torch.uint8).cuda()
    out, err = lhs.lhs_i8_matmul(lhs.lhs_i8_message(bad, m, k, response), tab)
    assert int(err.item()) == lhs.LHS_ERRBIT_MALFORMED
    assert bool(out[m - 1].isnan().all()) and same(out[:m - 1], ref[:m - 1])
    # a header that names another seq_len: every result is NaN
    bad = buf.clone() if not response else torch.cat([buf.new_zeros(4), buf])[4:]
    bad[4:8] = torch.tensor([m + 1], dtype=torch.int32).view(torch.uint8).cuda()
    out, err = lhs.lhs_i8_matmul(lhs.lhs_i8_message(bad, m, k, response), tab)
    assert int(err.item()) == lhs.LHS_ERRBIT_MALFORMED and bool(out.isnan().all())


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 12, 150])
def test_chain_on_another_stream(m):
    # table quantised, then multiplied, on a stream of its own; junk in the
    # buffers before each turn shows a read that ran ahead of its producer
    rng = np.random.default_rng(m)
    n, k = 20000, 640
    w = rng.standard_normal((n, k)).astype(np.float32)
    x = rng.standard_normal((m, k)).astype(np.float32)
    wq, wsc, _ = ref_quantize(w)
    xq, xsc, _ = ref_quantize(x)
    ref = ref_logits(xq, xsc, wq, wsc, torch.float32).cuda()
    wd, xd = torch.from_numpy(w).cuda(), torch.from_numpy(x).cuda()
    st = torch.cuda.Stream()
    codes = torch.empty((n, k), dtype=torch.int8, device="cuda")
    scales = torch.empty(n, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(lhs.lhs_i8_workspace(lhs.lhs_i8_init(codes, scales, k), m), dtype=torch.uint8, device="cuda")
    out = torch.empty((m, n), device="cuda")
    torch.cuda.synchronize()
    bad = 0
    for _ in range(30):
        with torch.cuda.stream(st):
            codes.fill_(85)
            scales.fill_(float("nan"))
            ws.fill_(0xFF)
            out.fill_(float("nan"))
            tab, _ = lhs.lhs_i8_quantize(wd, codes=codes, scales=scales, err=err, stream=st)
            lhs.lhs_i8_logits(tab, xd, out=out, ws=ws, err=err, stream=st)
        st.synchronize()
        bad += not torch.equal(out, ref)
    assert bad == 0 and int(err.item()) == 0


@pytest.mark.gpu
def test_captured_call_replays():
    rng = np.random.default_rng(8)
    wb, ws = make_rows(rng, 5000, 896)
    tab = table_of(wb, ws, 896)
    x = torch.zeros((4, 896), device="cuda")
    out = torch.empty((4, 5000), device="cuda")
    work = torch.empty(lhs.lhs_i8_workspace(tab, 4), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lhs.lhs_i8_logits(tab, x, out=out, ws=work, err=err)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lhs.lhs_i8_logits(tab, x, out=out, ws=work, err=err)
    for seed in range(3):
        xn = np.random.default_rng(seed).standard_normal((4, 896)).astype(np.float32)
        x.copy_(torch.from_numpy(xn))
        g.replay()
        q, s, _ = ref_quantize(xn)
        assert same(out, ref_logits(q, s, wb[:, :896], ws, torch.float32))


@pytest.mark.gpu
def test_offsets_pass_32_bits():
    # the table's bytes and the logits' elements lie beyond 2^31
    n, k, m = 1_100_000, 2048, 2200
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    codes = torch.zeros((n, k), dtype=torch.int8, device="cuda")
    codes[-1] = 1
    codes[-2, :7] = 3
    scales = torch.ones(n, device="cuda")
    x = torch.zeros((m, k), device="cuda")
    x[:, 0] = 127.0
    x[-1, 1] = -64.0
    out = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    _, err = lhs.lhs_i8_logits(lhs.lhs_i8_init(codes, scales, k), x, out=out)
    assert int(err.item()) == 0
    assert out[:-1, -2:].float().unique().tolist() == [127.0, 380.0]  # 381 is a tie in bf16
    assert out[-1, -2:].tolist() == [189.0, 63.0]
    assert bool((out[:, :-2] == 0).all())


@pytest.mark.gpu
def test_agrees_with_the_message_oracle():
    # the same codes as the wire oracle writes
    x = np.random.default_rng(2).standard_normal((6, 64)).astype(np.float32)
    buf, _ = orc.wire_encode(orc.WIRE_I8, x)
    pos = np.frombuffer(buf.tobytes()[16:], np.uint8).reshape(6, 72)
    t, _ = lhs.lhs_i8_quantize(torch.from_numpy(x).cuda())
    assert np.array_equal(t.codes.cpu().numpy(), pos[:, 8:].view(np.int8))
    assert np.array_equal(t.scales.cpu().numpy(), pos[:, :4].copy().view(np.float32)[:, 0])
