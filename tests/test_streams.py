"""Calls that are given a stream: what a call allocates or clears itself
(default outputs, workspaces, error words) belongs to that stream, whatever
the current stream is doing meanwhile."""
import pytest
import torch

import embedding_lookup_tied_gb300 as lhs

pytestmark = pytest.mark.gpu

V, H, N = 3000, 256, 64


@pytest.fixture(scope="module")
def data():
    g = torch.Generator().manual_seed(5)
    table = torch.randn((V, H), generator=g).cuda()
    x = torch.randn((N, H), generator=g).cuda()
    bad = x.clone()
    bad[3, 7] = float("nan")
    ids = torch.randint(0, V, (N,), generator=g, dtype=torch.int32).cuda()
    bad_ids = ids.clone()
    bad_ids[5] = V + 1
    head, _ = lhs.lhs_i8_quantize(table)
    tokens, _ = lhs.lhs_i8_quantize(x)
    logits = torch.randn((N, V), generator=g).cuda()
    bad_logits = logits.clone()
    bad_logits[2, 9] = float("inf")
    u = torch.rand(N, generator=g).cuda()
    wide = lhs.lhs_table_init(table, V, H, lhs.LHS_F32)
    msg = lhs.lhs_wire_encode(lhs.LHS_WIRE_I8, x)[0]
    resp = lhs.lhs_wire_encode_response(lhs.LHS_WIRE_I8, x)[0]
    bad_msg = msg.clone()
    bad_msg[4] ^= 1  # another seq_len
    raw = table.view(torch.uint8).reshape(-1)
    row_offset = torch.arange(V, dtype=torch.int64).cuda() * (4 * H)
    row_dtype = torch.full((V,), lhs.LHS_F32, dtype=torch.uint8).cuda()
    torch.cuda.synchronize()
    i8, f16 = lhs.LHS_WIRE_I8, lhs.LHS_WIRE_F16
    return {
        "i8_quantize": lambda **k: lhs.lhs_i8_quantize(x, **k),
        "i8_quantize_bad": lambda **k: lhs.lhs_i8_quantize(bad, **k),
        "i8_matmul": lambda **k: lhs.lhs_i8_matmul(tokens, head, **k),
        "i8_matmul_bad": lambda **k: lhs.lhs_i8_matmul(lhs.lhs_i8_message(bad_msg, N, H), head, **k),
        "i8_logits": lambda **k: lhs.lhs_i8_logits(head, x, **k),
        "i8_logits_bad": lambda **k: lhs.lhs_i8_logits(head, bad, **k),
        "i8_logits_few_bad": lambda **k: lhs.lhs_i8_logits(head, bad[:8], **k),
        "sample": lambda **k: lhs.lhs_sample(logits, u, **k),
        "sample_bad": lambda **k: lhs.lhs_sample(bad_logits, u, **k),
        "embed_bad": lambda **k: lhs.lhs_embed(wide, bad_ids, 1.0, **k),
        "embed_wire_bad": lambda **k: lhs.lhs_embed_wire(wide, bad_ids, 1.0, f16, **k),
        "embed_wire_response_bad": lambda **k: lhs.lhs_embed_wire_response(wide, bad_ids, 1.0, f16, **k),
        "unique_ids_bad": lambda **k: lhs.lhs_unique_ids(bad_ids, V, **k)[1:],
        "embed_dedup_bad": lambda **k: lhs.lhs_embed_dedup(wide, bad_ids, 1.0, **k),
        "embed_mixed_bad": lambda **k: lhs.lhs_embed_mixed(raw, row_offset, row_dtype, V, H, bad_ids, 1.0, **k),
        "logits_topk": lambda **k: lhs.lhs_logits_topk(wide, x[:4], 5, **k),
        "logits": lambda **k: lhs.lhs_logits(wide, x[:4], **k),
        "logits_topk_noalloc": lambda **k: lhs.lhs_logits_topk_noalloc(wide, x[:4], 5, **k),
        "wire_encode_bad": lambda **k: lhs.lhs_wire_encode(i8, bad, **k),
        "wire_decode": lambda **k: lhs.lhs_wire_decode(i8, msg, N, H, **k),
        "wire_encode_response_bad": lambda **k: lhs.lhs_wire_encode_response(i8, bad, **k),
        "wire_decode_response": lambda **k: lhs.lhs_wire_decode_response(i8, resp, N, H, **k),
    }


CALLS = ["i8_quantize", "i8_quantize_bad", "i8_matmul", "i8_matmul_bad", "i8_logits", "i8_logits_bad",
         "i8_logits_few_bad", "sample", "sample_bad", "embed_bad", "embed_wire_bad", "embed_wire_response_bad",
         "unique_ids_bad", "embed_dedup_bad", "embed_mixed_bad", "logits_topk", "logits", "logits_topk_noalloc",
         "wire_encode_bad", "wire_decode", "wire_encode_response_bad", "wire_decode_response"]


def parts(results):
    out = []
    for r in results:
        out += [r.codes, r.scales] if isinstance(r, lhs.I8Rows) else [] if r is None else [r]
    return out


def equal(a, b):
    a, b = a.cpu(), b.cpu()
    if a.is_floating_point():
        return a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())
    return torch.equal(a, b)


@pytest.mark.parametrize("as_int", [False, True], ids=["Stream", "handle"])
@pytest.mark.parametrize("name", CALLS)
def test_default_buffers_while_the_current_stream_is_busy(data, name, as_int):
    call = data[name]
    want = [t.clone() for t in parts(call())]
    if name.endswith("_bad"):
        assert int(want[-1].item()) != 0
    st = torch.cuda.Stream()
    for turn in range(2):
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # the current stream gets to nothing for some 10 ms
        got = parts(call(stream=st.cuda_stream if as_int else st))
        torch.cuda.synchronize()
        assert len(got) == len(want)
        for g, w in zip(got, want):
            assert equal(g, w), (name, turn)


def test_a_stream_may_be_given_by_position(data):
    g = torch.Generator().manual_seed(6)
    x = torch.randn((40, 128), generator=g).cuda()
    want = [t.clone() for t in parts(lhs.lhs_i8_quantize(x))]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    got = parts(lhs.lhs_i8_quantize(x, None, None, None, st))
    torch.cuda.synchronize()
    assert all(equal(a, b) for a, b in zip(got, want))


def test_default_stream_from_another(data):
    # the default stream's handle is 0
    want = [t.clone() for t in parts(data["i8_logits_bad"]())]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for st in (0, torch.cuda.default_stream()):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            got = parts(data["i8_logits_bad"](stream=st))
        torch.cuda.synchronize()
        assert all(equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["lhs_i8_logits", "lhs_i8_matmul", "lhs_logits_topk", "lhs_embed_dedup"])
def test_workspace_is_not_handed_out_again(name, monkeypatch):
    # the call's own workspace may be in use on its stream after the call has returned: an
    # allocation of the current stream must not get it
    g = torch.Generator().manual_seed(7)
    table = torch.randn((4000, 512), generator=g).cuda()
    x = torch.randn((64, 512), generator=g).cuda()
    head, tokens = lhs.lhs_i8_quantize(table)[0], lhs.lhs_i8_quantize(x)[0]
    half = lhs.lhs_table_init(table.to(torch.bfloat16), 4000, 512, lhs.LHS_BF16)
    ids = torch.arange(64, dtype=torch.int32, device="cuda")
    call = {"lhs_i8_logits": lambda st: lhs.lhs_i8_logits(head, x, stream=st),
            "lhs_i8_matmul": lambda st: lhs.lhs_i8_matmul(tokens, head, stream=st),
            "lhs_logits_topk": lambda st: lhs.lhs_logits_topk(half, x.to(torch.bfloat16), 5, stream=st),
            "lhs_embed_dedup": lambda st: lhs.lhs_embed_dedup(half, ids, 1.0, stream=st)}[name]
    at = {"lhs_i8_logits": 8, "lhs_i8_matmul": 5, "lhs_logits_topk": 9, "lhs_embed_dedup": 5}[name]
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
