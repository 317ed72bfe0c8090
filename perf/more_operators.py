"""The operators that score and train a tied table, in their plain form and through this package.

* ``loss``: softmax cross entropy of given targets over the whole vocabulary,
  from the residuals and the table (no logits are asked for), and the
  logarithm of the normaliser; 0 for tokens without a target.
* ``train``: the same with its gradient, for the residuals and for the table;
  where the case is ``tied``, the gradient of the tokens' lookups is added to
  the table's.
* ``embed``: the gradient of the scaled embedding lookup for the whole table.

``run`` takes the plain form where ``own`` is false and the package's entry
points where it is true.  ``exact`` is each operator in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
IGNORE = -100


def loss_case(name, t, v, h, dt, masked=0.0, temperature=1.0):
    """t tokens against a v x h table of type dt; masked: the part of the tokens without a target."""
    c = {"op": "loss", "t": t, "v": v, "h": h, "dt": dt, "masked": masked, "temperature": temperature}
    return {"name": name, **c} if name else c


def train_case(name, t, v, h, dt, masked=0.0, temperature=1.0, tied=False):
    c = {"op": "train", "t": t, "v": v, "h": h, "dt": dt, "masked": masked, "temperature": temperature, "tied": tied}
    return {"name": name, **c} if name else c


def embed_case(name, n, v, h, dout, dt):
    """n lookups, gradients of type dout, into a v x h gradient of type dt."""
    c = {"op": "embed", "n": n, "v": v, "h": h, "dout": dout, "dt": dt}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the smallest call: 16 tokens of the 8,192-word vocabulary; latency
        loss_case("loss-tiny-16", 16, 8192, 256, "bf16"),
        # the log-probability of one token over the 151,936 x 896 table: one stream of the table
        loss_case("loss-score-1", 1, 151936, 896, "bf16"),
        # scoring a 628-token session
        loss_case("loss-session-628", 628, 151936, 896, "bf16"),
        # scoring 2,048 tokens against the 262,144 x 5,376 table: the most work of a call
        loss_case("loss-batch-2048", 2048, 262144, 5376, "f16"),
        # odd sizes in every direction, prompts without targets, a temperature
        loss_case("loss-ragged-333", 333, 8191, 1001, "f16", 0.35, 0.7),
        # a training step of the smallest table
        train_case("train-tiny-64", 64, 8192, 256, "bf16"),
        # 256 tokens against the 262,144 x 5,120 table: the table's gradient dominates
        train_case("train-batch-256", 256, 262144, 5120, "bf16"),
        # a batch of 8,192 tokens, tied: the lookups' gradient joins the loss's
        train_case("train-tied-8192", 8192, 151936, 896, "bf16", 0.0, 1.0, True),
        # fine-tuning: half of the tokens are prompt or padding, f16 with a scaled loss
        train_case("train-masked-4096", 4096, 262144, 768, "f16", 0.5),
        # the smallest lookup's gradient
        embed_case("embed-tiny-16", 16, 8192, 256, "f32", "f32"),
        # 64 sequences of 128 tokens, 262,144 x 768
        embed_case("embed-8192", 8192, 262144, 768, "f32", "bf16"),
        # a large batch: hot tokens with tens of thousands of positions each
        embed_case("embed-large", 262144, 151936, 896, "bf16", "bf16"),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["loss", "train", "embed"])
    v, h = log_int(rng, 500, 262144), log_int(rng, 64, 5376)
    if rng.random() < 0.6:  # most tables have rows of whole 16-byte words
        h = h // 8 * 8
    if op == "embed":
        n = log_int(rng, 1, 262144)
        while n * h > 2.3e8 or v * h > 2.3e8:
            n, v = max(1, n * 3 // 4), max(500, v * 3 // 4)
        return embed_case("", n, v, h, rng.choice(["f32", "bf16", "f16"]), rng.choice(["f32", "bf16", "f16"]))
    t = log_int(rng, 1, 8192)
    most = 2.8e12 if op == "loss" else 1.1e12
    while t * v * h > most or v * h > 1.41e9 or t * v > 1.3e9:
        t, v = max(1, t * 4 // 5), max(500, v * 4 // 5)
    masked, temp = rng.choice([0.0, 0.0, 0.3, 0.6]), rng.choice([1.0, 1.0, 0.7, 1.5])
    dt = rng.choice(["bf16", "f16"])
    if op == "loss":
        return loss_case("", t, v, h, dt, masked, temp)
    return train_case("", t, v, h, dt, masked, temp, rng.random() < 0.4)


def active(case):
    """Tokens that have a target (at least one)."""
    return max(1, case["t"] - int(case["t"] * case["masked"]))


def zipf_ids(n, v, g, dev):
    """n ids, rank r with probability proportional to r^-1.1, ranks scattered over the vocabulary."""
    w = torch.arange(1, v + 1, dtype=torch.float64, device=dev) ** -1.1
    c = torch.cumsum(w, 0)
    u = torch.rand(n, generator=g, device=dev, dtype=torch.float64) * c[-1]
    rank = torch.searchsorted(c, u).clamp(max=v - 1)
    return torch.randperm(v, generator=g, device=dev)[rank].to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    s = dict(case)
    s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)  # the request's error word
    v, h = case["v"], case["h"]

    def rows_of(n, dt, lo, hi):  # Gaussian rows of different sizes
        x = torch.randn((n, h), generator=g, device=dev)
        x *= torch.rand((n, 1), generator=g, device=dev) * (hi - lo) + lo
        return x.to(DT[dt])

    if case["op"] == "embed":
        s["ids"] = zipf_ids(case["n"], v, g, dev)
        s["rows"] = rows_of(case["n"], case["dout"], 0.01, 1.0)
        s["scale"] = math.sqrt(h)
        return s
    t = case["t"]
    table = torch.empty((v, h), dtype=DT[case["dt"]], device=dev)
    for r in range(0, v, 32768):
        table[r:r + 32768] = (torch.randn((min(32768, v - r), h), generator=g, device=dev) * 0.02).to(table.dtype)
    s["table"] = table
    y = zipf_ids(t, v, g, dev)
    # logits from almost flat to peaked; the target's from unlikely to nearly certain, as a model in training has them
    x = torch.randn((t, h), generator=g, device=dev)
    x *= (torch.rand((t, 1), generator=g, device=dev) * 4.0 + 0.5) / (0.02 * math.sqrt(h))
    x *= 0.5
    w = table[y.long()].float()
    x += w * (torch.rand((t, 1), generator=g, device=dev) * 14.0 / (w * w).sum(1, keepdim=True).clamp(min=1e-6))
    s["x"] = x.to(table.dtype)
    off = torch.randperm(t, generator=g, device=dev)[active(case):]
    y[off] = IGNORE
    s["targets"] = y
    if case["op"] == "train":
        # a mean over the tokens with a weight each; f16 gradients need a scaled loss
        s["dloss"] = (torch.rand(t, generator=g, device=dev) + 0.5) / active(case)
        if case["dt"] == "f16":
            s["dloss"] *= 8192.0
        if case["tied"]:
            s["ids"] = zipf_ids(t, v, g, dev)
            s["rows"] = rows_of(t, case["dt"], 0.01, 1.0)
            s["rows"] *= s["dloss"].max()
            s["scale"] = math.sqrt(h)
    return s


def run(state):
    return (own_run if own else plain_run)(state)


def own_run(s):
    import embedding_lookup_tied_gb300 as lhs
    if s["op"] == "embed":
        return lhs.lhs_embed_grad(s["ids"], s["rows"], s["v"], s["scale"], dtype=DT[s["dt"]], err=s["err"])[0]
    table = lhs.lhs_table_init(s["table"], s["v"], s["h"], lhs.LHS_BF16 if s["dt"] == "bf16" else lhs.LHS_F16)
    loss, lse, _ = lhs.lhs_loss(table, s["x"], s["targets"], temperature=s["temperature"], err=s["err"])
    if s["op"] == "loss":
        return {"loss": loss, "lse": lse}
    dx, dtable, _ = lhs.lhs_loss_grad(table, s["x"], s["targets"], lse, s["dloss"], temperature=s["temperature"],
                                      err=s["err"])
    if s["tied"]:
        lhs.lhs_embed_grad(s["ids"], s["rows"], s["v"], s["scale"], dtable=dtable, accumulate=True, err=s["err"])
    return {"loss": loss, "dx": dx, "dtable": dtable}


def plain_run(s):
    if s["op"] == "embed":
        return plain_lookup_grad(s).to(DT[s["dt"]])
    y = s["targets"].long()
    on = y != IGNORE
    x, w, y = s["x"][on].float(), s["table"].float(), y[on][:, None]
    z = x @ w.T
    z /= s["temperature"]
    top = z.amax(1, keepdim=True)
    at = z.gather(1, y)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    loss = torch.zeros((2, len(on)), device=x.device)
    loss[:, on] = torch.stack([(lse - at)[:, 0], lse[:, 0]])
    if s["op"] == "loss":
        return {"loss": loss[0], "lse": loss[1]}
    g = z.sub_(lse).exp_()
    g.scatter_add_(1, y, torch.full_like(at, -1.0))
    g *= (s["dloss"][on] / s["temperature"])[:, None]
    dx = torch.zeros_like(s["x"])
    dx[on] = (g @ w).to(dx.dtype)
    dw = g.T @ x
    if s["tied"]:
        dw = dw.double() + plain_lookup_grad(s)
    return {"loss": loss[0], "dx": dx, "dtable": dw.to(s["table"].dtype)}


def plain_lookup_grad(s):
    d = torch.zeros((s["v"], s["h"]), dtype=torch.float64, device=s["ids"].device)  # long sums
    d.index_add_(0, s["ids"].long(), s["rows"].double())
    return d.mul_(s["scale"])


def exact(case, seed):
    if case["op"] != "embed":
        flops = (2 if case["op"] == "loss" else 6) * active(case) * case["v"] * case["h"]
        if flops > 1.2e13:
            return None
    s = prepare(case, seed)
    if case["op"] == "embed":
        return exact_lookup_grad(s)
    t, v, h, temp = case["t"], case["v"], case["h"], case["temperature"]
    w = s["table"].double()
    loss, lse = np.zeros(t), np.zeros(t)
    train = case["op"] == "train"
    if train:
        dx = torch.zeros((t, h), dtype=torch.float64, device="cuda")
        dw = torch.zeros((v, h), dtype=torch.float64, device="cuda")
    with_target = np.flatnonzero(s["targets"].cpu().numpy() != IGNORE)
    for r in range(0, len(with_target), 1024):
        at = torch.from_numpy(with_target[r:r + 1024]).cuda()
        xs, ys = s["x"].index_select(0, at).double(), s["targets"].index_select(0, at).long()
        z = torch.mm(xs, w.t()).div_(temp)
        norm = torch.logsumexp(z, dim=1)
        one = torch.arange(len(at), device="cuda")
        loss[with_target[r:r + 1024]] = (norm - z[one, ys]).cpu().numpy()
        lse[with_target[r:r + 1024]] = norm.cpu().numpy()
        if train:
            p = torch.exp(z - norm[:, None])
            p[one, ys] = torch.expm1(z[one, ys] - norm)
            p.mul_(s["dloss"].index_select(0, at).double()[:, None] / temp)
            dx.index_copy_(0, at, torch.mm(p, w))
            dw.addmm_(p.t(), xs)
    if not train:
        return {"loss": loss, "lse": lse}
    if case["tied"]:
        dw += exact_lookup_grad(s)
    return {"loss": loss, "dx": dx, "dtable": dw}


def exact_lookup_grad(s):
    """Sums over the positions of each id, positions in order."""
    ids = s["ids"].cpu().numpy()
    order = np.argsort(ids, kind="stable")
    first = np.flatnonzero(np.r_[True, np.diff(ids[order]) != 0])
    out = torch.zeros((s["v"], s["h"]), dtype=torch.float64, device="cuda")
    where = torch.from_numpy(ids[order][first].astype(np.int64)).cuda()
    for j in range(0, s["h"], 128):
        part = s["rows"][:, j:j + 128].double().cpu().numpy()[order]
        sums = np.add.reduceat(part, first, axis=0) * s["scale"]
        out[:, j:j + 128].index_copy_(0, where, torch.from_numpy(sums).cuda())
    return out


def work(case):
    v, h = case["v"], case["h"]
    if case["op"] == "embed":
        n = case["n"]
        # the gradients and ids once, the table's gradient once; one addition a value
        return {"bytes": n * (h * SIZE[case["dout"]] + 4) + v * h * SIZE[case["dt"]], "flops": n * h}
    t, a, e = case["t"], active(case), SIZE[case["dt"]]
    size = v * h * e + a * h * e + 8 * t
    if case["op"] == "loss":
        return {"bytes": size, "flops": 2 * a * v * h}
    size += v * h * e + t * h * e + 4 * t + (t * (h * e + 4) if case["tied"] else 0)
    # the logits and two products of the same size
    return {"bytes": size, "flops": 6 * a * v * h}
