"""Two operators of a quantised decode step, in their plain form and through this package.

* ``i8``: the tied lm_head as a matrix product in 8-bit integers, with one
  scale for each token and one for each channel (vocabulary row).  A token
  arrives either wide (f32, bf16 or f16 residuals, quantised per token within
  the pass) or as a position of an i8 residual message (its scale, a zero
  point and its codes).
* ``sample``: one token per row of logits, drawn with temperature, top-k,
  top-p and min-p from a given random number.

``run`` takes the plain form where ``own`` is false and the package's entry
points where it is true.  ``exact`` is either operator in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def i8_case(name, m, n, k, x, out):
    """m tokens against n channels of k codes; x: the tokens' form; out: the logits' type."""
    c = {"op": "i8", "m": m, "n": n, "k": k, "x": x, "out": out}
    return {"name": name, **c} if name else c


def sample_case(name, b, v, t, mode, masked=False):
    """b rows of v logits of type t; mode: which filters the rows use; masked: some rows
    allow part of the vocabulary only."""
    c = {"op": "sample", "b": b, "v": v, "t": t, "mode": mode, "masked": masked}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one sequence's decode step over the 151,936 x 896 table: latency, one stream of the codes
        i8_case("i8-decode-1", 1, 151936, 896, "f32", "f32"),
        # eight sequences over the 262,144 x 5,376 table: as much HBM traffic as a step can have
        i8_case("i8-decode-8", 8, 262144, 5376, "f32", "f32"),
        # 256 sequences over the 262,144 x 5,120 table: the largest batch, tensor-core work
        i8_case("i8-batch-256", 256, 262144, 5120, "bf16", "f32"),
        # the logits of a whole 628-token session (scoring a prompt)
        i8_case("i8-session-628", 628, 151936, 896, "bf16", "bf16"),
        # 64 residuals straight out of an i8 message, 262,144 x 768 table
        i8_case("i8-message-64", 64, 262144, 768, "message", "f16"),
        # odd sizes: ragged in every direction, a vocabulary of 8,191
        i8_case("i8-ragged-37", 37, 8191, 1001, "f16", "bf16"),
        # the smallest call: four rows of the 8,192-word vocabulary
        sample_case("sample-tiny-4", 4, 8192, "f32", "all"),
        # one sequence's decode step with the usual filters
        sample_case("sample-decode-1", 1, 151936, "f32", "all"),
        # eight sequences, nucleus only: the threshold lies deep in the row
        sample_case("sample-nucleus-8", 8, 262144, "f32", "top_p"),
        # the largest batch, every row with filters of its own, grammar masks on some rows
        sample_case("sample-batch-256", 256, 262144, "f32", "mixed", True),
        # min-p alone on 16-bit logits (many equal values)
        sample_case("sample-minp-64", 64, 151936, "bf16", "min_p"),
        # odd sizes, 16-bit rows that start at every alignment, masks
        sample_case("sample-ragged-37", 37, 8191, "f16", "mixed", True),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        m, n, k = log_int(rng, 1, 640), log_int(rng, 500, 262144), log_int(rng, 64, 5376)
        x = rng.choice(["f32", "bf16", "f16", "message"])
        if x == "message":
            k = max(64, k - k % 4)  # positions of k + 8 bytes start on 4-byte boundaries
        while 2 * m * n * k > 6.8e11 or n * k > 1.4e9 or m * n > 9e7:
            n = max(500, n * 3 // 4)
        return i8_case("", m, n, k, x, rng.choice(["f32", "bf16", "f16"]))
    b, v = log_int(rng, 1, 256), log_int(rng, 1000, 262144)
    return sample_case("", b, v, rng.choice(["f32", "bf16", "f16"]),
                       rng.choice(["all", "top_k", "top_p", "min_p", "plain", "mixed"]), rng.random() < 0.3)


def codes_of(x):
    """Symmetric 8-bit codes of f32 rows: scale = max|x| / 127, code = x / scale rounded to the
    nearest integer, ties to even; an all-zero row has scale 0 and codes 0."""
    top = x.abs().amax(1)
    scale = top / torch.full_like(top, 127.0)  # a correctly rounded quotient (a plain number would be multiplied by its inverse)
    code = torch.round(x / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]).clamp(-127, 127)
    return code, scale


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    s = dict(case)
    s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)  # the request's error word
    if case["op"] == "i8":
        m, n, k = case["m"], case["n"], case["k"]
        # the table, quantised once when it was loaded: rows of k codes on 16-byte boundaries
        codes = torch.zeros((n, (k + 15) // 16 * 16), dtype=torch.int8, device=dev)
        scales = torch.empty(n, dtype=torch.float32, device=dev)
        for r in range(0, n, 32768):
            w = torch.randn((min(32768, n - r), k), generator=g, device=dev) * 0.02
            q, sc = codes_of(w)
            codes[r:r + len(w), :k] = q.to(torch.int8)
            scales[r:r + len(w)] = sc
        x = torch.randn((m, k), generator=g, device=dev)
        x *= torch.rand((m, 1), generator=g, device=dev) * 7.5 + 0.5
        s["codes"], s["scales"] = codes, scales
        if case["x"] == "message":
            q, sc = codes_of(x)
            head = torch.tensor([0, m, 0, 10], dtype=torch.int32, device=dev).view(torch.uint8)
            rows = torch.cat([sc[:, None].contiguous().view(torch.uint8),
                              torch.zeros((m, 4), dtype=torch.uint8, device=dev),
                              q.to(torch.int8).view(torch.uint8)], 1)
            s["msg"] = torch.cat([head, rows.reshape(-1)])
        else:
            s["x"] = x.to(DT[case["x"]])
        return s
    b, v, mode = case["b"], case["v"], case["mode"]
    logits = torch.randn((b, v), generator=g, device=dev)
    # rows from almost flat to peaked, with a few tokens that stand out
    logits *= torch.rand((b, 1), generator=g, device=dev) * 4.0 + 0.7
    few = torch.randint(0, v, (b, 8), generator=g, device=dev)
    logits.scatter_add_(1, few, torch.rand((b, 8), generator=g, device=dev) * 8.0)
    if case["masked"]:  # every third row may use some of the vocabulary only
        rows = torch.arange(b, device=dev) % 3 == 1
        some = torch.rand((b, v), generator=g, device=dev) < 0.9
        logits.masked_fill_(some & rows[:, None], float("-inf"))
    s["logits"] = logits.to(DT[case["t"]])
    s["u"] = torch.rand(b, generator=g, device=dev)

    def pick(lo, hi):
        return torch.rand(b, generator=g, device=dev) * (hi - lo) + lo

    # None: the filter is off for every row
    s["temperature"] = pick(0.6, 1.3)
    s["top_k"] = torch.randint(20, 200, (b,), generator=g, device=dev, dtype=torch.int32) if mode in ("all", "top_k", "mixed") else None
    s["top_p"] = pick(0.8, 0.98) if mode in ("all", "top_p", "mixed") else None
    s["min_p"] = pick(0.01, 0.1) if mode in ("all", "min_p", "mixed") else None
    if mode == "mixed":  # rows of different requests: any filter may be off, some rows are greedy
        kind = torch.randint(0, 8, (b,), generator=g, device=dev)
        s["temperature"] = torch.where(kind == 0, torch.zeros_like(s["temperature"]), s["temperature"])
        s["top_k"] = torch.where(kind % 2 == 1, torch.zeros_like(s["top_k"]), s["top_k"])
        s["top_p"] = torch.where(kind >= 5, torch.ones_like(s["top_p"]), s["top_p"])
        s["min_p"] = torch.where((kind == 2) | (kind == 5) | (kind == 7), torch.zeros_like(s["min_p"]), s["min_p"])
    return s


def run(state):
    if state["op"] == "i8":
        return own_i8(state) if own else plain_i8(state)
    return own_sample(state) if own else plain_sample(state)


def own_i8(s):
    import embedding_lookup_tied_gb300 as lhs
    table = lhs.lhs_i8_init(s["codes"], s["scales"], s["k"])
    if s["x"] == "message":
        tokens = lhs.lhs_i8_message(s["msg"], s["m"], s["k"])
        return lhs.lhs_i8_matmul(tokens, table, out_dtype=DT[s["out"]], err=s["err"])[0]
    return lhs.lhs_i8_logits(table, s["x"], out_dtype=DT[s["out"]], err=s["err"])[0]


def own_sample(s):
    import embedding_lookup_tied_gb300 as lhs
    ids, probs, _ = lhs.lhs_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                   top_p=s["top_p"], min_p=s["min_p"], err=s["err"])
    return {"ids": ids, "probs": probs}


def plain_i8(s):
    m, k = s["m"], s["k"]
    if s["x"] == "message":
        rows = s["msg"][16:].view(m, k + 8)
        scale = rows[:, :4].contiguous().view(torch.float32)[:, 0]
        code = rows[:, 8:].contiguous().view(torch.int8).float()
    else:
        code, scale = codes_of(s["x"].float())
    acc = code @ s["codes"][:, :k].float().T
    return (acc * scale[:, None] * s["scales"][None, :]).to(DT[s["out"]])


def plain_sample(s):
    x = s["logits"].double()
    b, v = x.shape
    col = lambda t, off: torch.full((b, 1), off, dtype=torch.float64, device=x.device) if t is None else t.double()[:, None]  # noqa: E731
    t, k, p, q = col(s["temperature"], 1.0), col(s["top_k"], 0.0), col(s["top_p"], 1.0), col(s["min_p"], 0.0)
    greedy = t == 0
    t, k = torch.where(greedy, 1.0, t), torch.where(greedy, 1.0, k)
    k = torch.where((k <= 0) | (k > v), float(v), k)
    z, order = torch.sort(x, dim=1, descending=True, stable=True)  # equal logits: the lowest id first
    w = torch.exp((z - z[:, :1]) / t)
    w = torch.where(torch.arange(v, device=x.device)[None, :] < k, w, 0.0)  # the k largest
    before = torch.cumsum(w, 1) - w
    keep = (before < p * w.sum(1, keepdim=True)) | (p >= 1)  # the shortest head whose mass reaches p of theirs
    w = torch.where(keep & (w >= q), w, 0.0)  # min-p: against the largest weight, which is 1
    w = torch.zeros_like(w).scatter_(1, order, w)  # back to id order
    c = torch.cumsum(w, 1)
    at = (c <= s["u"].double()[:, None] * c[:, -1:]).sum(1, keepdim=True)  # the first id whose running mass passes u
    return {"ids": at[:, 0].to(torch.int32), "probs": (w.gather(1, at)[:, 0] / c[:, -1]).float()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "i8":
        m, k = case["m"], case["k"]
        if case["x"] == "message":
            raw = s["msg"].cpu().numpy()[16:].reshape(m, k + 8)
            a_scale = np.ascontiguousarray(raw[:, :4]).view(np.float32)[:, 0].astype(np.float64)
            a = np.ascontiguousarray(raw[:, 8:]).view(np.int8).astype(np.float64)
        else:  # the codes are defined on scales and quotients of 32 bits: 64-bit quotients, rounded once
            x = s["x"].double().cpu().numpy()
            a_scale = (np.abs(x).max(1) / 127.0).astype(np.float32).astype(np.float64)
            quot = (x / np.where(a_scale > 0, a_scale, 1.0)[:, None]).astype(np.float32)
            a = np.clip(np.rint(quot), -127, 127).astype(np.float64)
        a, a_scale = torch.from_numpy(a).cuda(), torch.from_numpy(a_scale).cuda()
        out = torch.empty((m, case["n"]), dtype=torch.float64, device="cuda")
        for r in range(0, case["n"], 32768):  # sums of integers: exact in 64 bits
            w = s["codes"][r:r + 32768, :k].double()
            out[:, r:r + 32768] = torch.mm(a, w.t()) * torch.outer(a_scale, s["scales"][r:r + 32768].double())
        return out
    x = s["logits"].double().cpu().numpy()
    get = lambda t, off: np.full(case["b"], off) if t is None else t.double().cpu().numpy()  # noqa: E731
    temp, top_k, top_p, min_p = get(s["temperature"], 1.0), get(s["top_k"], 0), get(s["top_p"], 1.0), get(s["min_p"], 0.0)
    u = s["u"].double().cpu().numpy()
    ids, probs = [], []
    for r in range(case["b"]):
        row = x[r]
        if temp[r] == 0:
            ids.append(int(np.argmax(row)))
            probs.append(1.0)
            continue
        e = np.exp((row - row.max()) / temp[r])
        cand = np.flatnonzero(e > 0)
        if 0 < top_k[r] < len(cand):
            k = int(top_k[r])
            edge = np.partition(row[cand], len(cand) - k)[len(cand) - k]
            above = cand[row[cand] > edge]
            cand = np.sort(np.concatenate([above, cand[row[cand] == edge][:k - len(above)]]))
        if top_p[r] < 1:
            by = cand[np.argsort(-row[cand], kind="stable")]
            mass = np.cumsum(e[by])
            cand = np.sort(by[:int(np.searchsorted(mass, top_p[r] * mass[-1], side="left")) + 1])
        cand = cand[e[cand] >= min_p[r]]
        mass = np.cumsum(e[cand])
        at = cand[int(np.searchsorted(mass, u[r] * mass[-1], side="right"))]
        ids.append(int(at))
        probs.append(e[at] / mass[-1])
    return {"ids": np.array(ids, dtype=np.int32), "probs": np.array(probs)}


def work(case):
    if case["op"] == "i8":
        m, n, k = case["m"], case["n"], case["k"]
        tokens = m * (k + 8) if case["x"] == "message" else m * k * SIZE[case["x"]]
        return {"bytes": n * (k + 4) + tokens + m * n * SIZE[case["out"]], "flops": 2 * m * n * k}
    b, v = case["b"], case["v"]
    # the logits once, five parameters and two results a row; a difference and a comparison for each logit
    return {"bytes": b * v * SIZE[case["t"]] + 28 * b, "flops": 2 * b * v}
