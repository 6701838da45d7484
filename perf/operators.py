"""The training operators of the n-gram memory and its connection, measured case by case.

Five operators, each called as a training or serving program calls it:

  embed     engram_embed            rows of a table looked up by id, scaled, optionally summed per token
  grad      engram_embed_grad       the table's gradient by sorted ids, every row written
            engram_embed_grad_rows  the same for tables too large for a dense gradient: distinct ids and their rows
  quant     engram_fp8_quantise     e4m3 values with one power-of-two scale per block of 128
  matmul    engram_fp8_matmul       the product of two such operands
  gate      engram_gate_add_grad    the backward pass of the gated add into the four streams

`run` calls them where `own` is true; elsewhere it computes the same in elementary
torch operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

VOCAB = 129280   # tokenizer vocabulary of the synthetic workloads
HIDDEN = 4096    # hidden size of the streams
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}
BYTES = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one slot: the call's latency
        {"name": "embed_one_token", "op": "embed", "T": 1, "R": 1, "D": HIDDEN, "rows": VOCAB,
         "table": "bf16", "out": "bf16", "pooled": False, "ids": "zipf", "dead": 0.0, "scale": 64.0},
        # the connection's 3 orders x 8 heads of 256-wide rows for a full prefill, 5 % dead tokens
        {"name": "embed_ngram_rows", "op": "embed", "T": 65536, "R": 24, "D": 256, "rows": 8000009,
         "table": "bf16", "out": "bf16", "pooled": False, "ids": "ngram", "dead": 0.05, "scale": 0.5},
        # a unit test's size: 256 tokens, 2 heads, rows of 256 summed per token, bf16 gradient
        {"name": "grad_tiny_pooled", "op": "grad", "T": 256, "R": 6, "D": 256, "rows": 4096,
         "dy": "bf16", "out": "bf16", "pooled": True, "sparse": False, "ids": "ngram", "dead": 0.0,
         "scale": 1.0 / 6},
        # the token embedding's dense fp32 gradient of a 16k-token step
        {"name": "grad_vocab_dense", "op": "grad", "T": 16384, "R": 1, "D": HIDDEN, "rows": VOCAB,
         "dy": "bf16", "out": "f32", "pooled": False, "sparse": False, "ids": "zipf", "dead": 0.0,
         "scale": 64.0},
        # the released table's gradient of a full prefill: 1.57 million ids in 384 million rows
        {"name": "grad_ngram_rows", "op": "grad", "T": 65536, "R": 24, "D": 256, "rows": 384006168,
         "dy": "bf16", "out": "f32", "pooled": False, "sparse": True, "ids": "ngram", "dead": 0.05,
         "scale": 0.5},
        # the concatenated rows of a few decode slots, before their projection
        {"name": "quant_decode", "op": "quant", "M": 37, "K": 6144, "x": "bf16", "block_rows": 1,
         "cols": False, "values": "rows"},
        # the projection's output gradient, for both of the products that read it
        {"name": "quant_both", "op": "quant", "M": 65536, "K": HIDDEN, "x": "f32", "block_rows": 1,
         "cols": True, "values": "grad"},
        # the projection of 16 decode slots: the weights are read once
        {"name": "matmul_decode", "op": "matmul", "M": 16, "N": HIDDEN, "K": 6144, "b_block": 128,
         "out": "f32", "a": "rows", "b": "weights"},
        # the projection of a full prefill
        {"name": "matmul_forward", "op": "matmul", "M": 65536, "N": HIDDEN, "K": 6144, "b_block": 128,
         "out": "f32", "a": "rows", "b": "weights"},
        # the weight gradient over a ragged batch of tokens
        {"name": "matmul_weight_grad", "op": "matmul", "M": HIDDEN, "N": 6144, "K": 16411, "b_block": 1,
         "out": "f32", "a": "grad", "b": "rows"},
        # the gate's backward pass: one step of 512 slots, and a full prefill with dead tokens
        {"name": "gate_512", "op": "gate", "T": 512, "D": HIDDEN, "dk": "f32", "dead": 0.0},
        {"name": "gate_prefill", "op": "gate", "T": 65536, "D": HIDDEN, "dk": "f32", "dead": 0.05},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step):
    """A width in [lo, hi]: mostly a multiple of `step`, sometimes any."""
    w = _log(rng, lo, hi)
    if rng.random() < 0.7:
        w = max(step, w // step * step)
    return w + 16 if w == 3 << 10 else w


def draw(rng):
    op = rng.choice(["embed", "grad", "grad", "quant", "matmul", "matmul", "gate"])
    if op in ("embed", "grad"):
        R = rng.choice([1, 1, 2, 6, 9, 24])
        D = _width(rng, 16, HIDDEN, 16)
        most = 65536 * 24 * 256 // (4 if op == "embed" else 2)
        T = _log(rng, 1, max(1, min(65536, most // (R * D))))
        rows = _log(rng, 100, max(200, min(8000009, (1 << 31) // D)))
        c = {"op": op, "T": T, "R": R, "D": D, "rows": rows, "out": rng.choice(["bf16", "f32"]),
             "pooled": R > 1 and rng.random() < 0.4, "ids": "ngram" if R > 1 else "zipf",
             "dead": rng.choice([0.0, 0.0, 0.1, 1.0 if T < 4 else 0.3]),
             "scale": rng.choice([1.0, 1.0 / R, math.sqrt(D)])}
        if op == "embed":
            c["table"] = rng.choice(["bf16", "f32"])
        else:
            c["dy"] = rng.choice(["bf16", "f32"])
            c["sparse"] = rng.random() < 0.5
            if not c["sparse"]:
                c["rows"] = min(rows, max(1, VOCAB * HIDDEN // D // 2))
        return c
    if op == "quant":
        K = _width(rng, 16, 8192, 128)
        return {"op": op, "M": _log(rng, 1, 65536 * HIDDEN // K // 2), "K": K, "x": rng.choice(["bf16", "f32"]),
                "block_rows": rng.choice([1, 1, 128]), "cols": rng.random() < 0.5,
                "values": rng.choice(["rows", "grad", "weights"])}
    if op == "matmul":
        N, K = _width(rng, 64, 8192, 128), _width(rng, 128, 16384, 128)
        M = _log(rng, 1, max(1, min(65536, 65536 * HIDDEN * 6144 // (N * K) // 4)))
        return {"op": op, "M": M + 1 if M == 3 << 10 else M, "N": N, "K": K, "b_block": rng.choice([1, 128]),
                "out": rng.choice(["bf16", "f32"]), "a": rng.choice(["rows", "grad"]), "b": rng.choice(["rows", "weights"])}
    D = max(16, _log(rng, 16, 8192) // 16 * 16)
    D = D + 16 if D == 3 << 10 else D
    return {"op": op, "T": _log(rng, 1, min(65536, 65536 * HIDDEN // D // 2)), "D": D,
            "dk": rng.choice(["bf16", "f32"]), "dead": rng.choice([0.0, 0.1])}


def _distinct(c):
    """About how many distinct ids a case has (measured on such inputs; for work())."""
    n = c["T"] * c["R"] * (1 - c["dead"])
    if c["ids"] == "zipf":
        share = min(1.0, 1.35 * max(n, 1) ** -0.165)
        return min(n * share, c["rows"])
    n *= 0.87 if c["T"] > 4096 else 0.95
    return c["rows"] * (1 - math.exp(-n / c["rows"]))


def work(c):
    op = c["op"]
    if op == "embed":
        n = c["T"] * c["R"]
        y = c["T"] if c["pooled"] else n
        return {"bytes": 4 * n + _distinct(c) * c["D"] * BYTES[c["table"]] + y * c["D"] * BYTES[c["out"]],
                "flops": n * c["D"]}
    if op == "grad":
        n = c["T"] * c["R"]
        dy = (c["T"] if c["pooled"] else n) * (1 - c["dead"])
        out = _distinct(c) if c["sparse"] else c["rows"]
        return {"bytes": 4 * n + dy * c["D"] * BYTES[c["dy"]] + out * c["D"] * BYTES[c["out"]]
                + (4 * out if c["sparse"] else 0), "flops": n * c["D"]}
    if op == "quant":
        n = c["M"] * c["K"]
        return {"bytes": n * BYTES[c["x"]] + (2 if c["cols"] else 1) * (n + n / 128 / c["block_rows"]), "flops": n}
    if op == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        kb = (K + 127) // 128
        return {"bytes": M * K + N * K + M * kb + N * kb / c["b_block"] + M * N * BYTES[c["out"]],
                "flops": 2 * M * N * K}
    T, D = c["T"], c["D"]
    return {"bytes": T * D * (4 + 2 + 8 + 8 + BYTES[c["dk"]]) + T + 16, "flops": 40 * T * D}


# -------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _zipf(g, n, most):
    """Zipf(1.1) ranks 0 .. most-1, as token ids of running text are spread."""
    w = torch.arange(1, most + 1, device="cuda", dtype=torch.float64) ** -1.1
    c = torch.cumsum(w, 0)
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * c[-1]
    return torch.searchsorted(c, u).clamp_(max=most - 1)


def _ids(c, g):
    """int32 [T, R] row ids: tokens by rank, or the 2-, 3- and 4-gram hashes of a text;
    a share of the tokens is dead (-1)."""
    T, R, rows = c["T"], c["R"], c["rows"]
    if c["ids"] == "zipf":
        ids = _zipf(g, T * R, rows).reshape(T, R)
    else:
        tok = torch.cat([torch.zeros(3, device="cuda", dtype=torch.int64), _zipf(g, T, VOCAB) + 1])
        cols = []
        for r in range(R):
            n = 2 + r * 3 // R
            h = torch.full((T,), 1000003 * (r + 1), device="cuda", dtype=torch.int64)
            for i in range(n):
                h = (h ^ tok[3 - i:3 - i + T]) * 0x1E3779B97F4A7C15
                h = h ^ ((h >> 29) & 0x7FFFFFFFF)
            cols.append((h & 0x3FFFFFFFFFFFFFFF) % rows)
        ids = torch.stack(cols, 1)
    if c["dead"] > 0:
        ids = torch.where(_rand(g, T, 1) < c["dead"], -1, ids)
    return ids.to(torch.int32).contiguous()


def _values(kind, g, M, K):
    """fp32 [M, K] as the path has them: concatenated table rows (blocks of 32 columns
    with scales 2^-10 .. 2^-7), gradients (a size of its own for each row), weights."""
    x = _randn(g, M, K)
    if kind == "rows":
        e = torch.randint(-10, -6, (M, (K + 31) // 32), generator=g, device="cuda").float()
        x *= torch.exp2(e).repeat_interleave(32, 1)[:, :K]
        x = torch.where(_rand(g, M, 1) < 0.02, 0.0, x)  # dead tokens
    elif kind == "grad":
        x *= 1e-4 * torch.exp(_randn(g, M, 1))
    else:
        x *= 2.0
    return x


def _blocks(x, br):
    """The largest magnitude of each block of br rows x 128 columns."""
    M, K = x.shape
    pm, pk = -M % br, -K % 128
    a = torch.nn.functional.pad(x.abs(), (0, pk, 0, pm))
    return a.reshape((M + pm) // br, br, (K + pk) // 128, 128).amax((1, 3))


def _spread(s, br, M, K):
    """A value per block as one per element."""
    if br > 1:
        s = s.repeat_interleave(br, 0)[:M]
    return s.repeat_interleave(128, 1)[:, :K]


def _quantise(x, br):
    """(e4m3 bytes [M, K], exponent bytes per block): the smallest power of two 2^(e-127)
    with every magnitude of the block at most 448 times it."""
    x = x.float()
    bits = _blocks(x, br).view(torch.int32)
    e = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000)).clamp_(0, 254)
    q = (x * torch.exp2(127.0 - _spread(e, br, *x.shape))).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), e.to(torch.uint8)


def _padded(q):
    """The bytes with rows a multiple of 16 apart."""
    M, K = q.shape
    p = torch.zeros(M, (K + 15) // 16 * 16, device="cuda", dtype=torch.uint8)
    p[:, :K] = q
    return p[:, :K]


def _empty_q(M, K):
    return torch.empty(M, (K + 15) // 16 * 16, device="cuda", dtype=torch.uint8)[:, :K]


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    s = {"case": c}
    if op == "embed":
        s["table"] = (_randn(g, c["rows"], c["D"]) * 0.02).to(DTYPES[c["table"]])
        s["ids"] = _ids(c, g)
        shape = (c["T"], c["D"]) if c["pooled"] else (c["T"], c["R"], c["D"])
        s["out"] = torch.empty(shape, device="cuda", dtype=DTYPES[c["out"]])
    elif op == "grad":
        s["ids"] = _ids(c, g)
        n = c["T"] * c["R"]
        shape = (c["T"], c["D"]) if c["pooled"] else (c["T"], c["R"], c["D"])
        s["dy"] = (_values("grad", g, math.prod(shape[:-1]), c["D"]).reshape(shape) * 10).to(DTYPES[c["dy"]])
        if c["sparse"]:
            s["row_ids"] = torch.full((n,), -1, device="cuda", dtype=torch.int32)
            s["grads"] = torch.zeros(n, c["D"], device="cuda", dtype=DTYPES[c["out"]])
            s["count"] = torch.zeros(1, device="cuda", dtype=torch.int32)
        else:
            s["grad"] = torch.empty(c["rows"], c["D"], device="cuda", dtype=DTYPES[c["out"]])
        # scratch as the library's own query states it, at most: 32 bytes an id and two
        # fp32 rows for every 16 ids, and 4 MB
        s["workspace"] = torch.empty(n * 32 + (n // 16 + 2) * 2 * (c["D"] + 8) * 4 + (4 << 20), device="cuda",
                                     dtype=torch.uint8)
    elif op == "quant":
        s["x"] = _values(c["values"], g, c["M"], c["K"]).to(DTYPES[c["x"]])
        br, M, K = c["block_rows"], c["M"], c["K"]
        s["q"] = [_empty_q(M, K), torch.empty(-(-M // br), -(-K // 128), device="cuda", dtype=torch.uint8)]
        if c["cols"]:
            s["q"] += [_empty_q(K, M), torch.empty(-(-K // br), -(-M // 128), device="cuda", dtype=torch.uint8)]
    elif op == "matmul":
        q, s["a_scale"] = _quantise(_values(c["a"], g, c["M"], c["K"]), 1)
        s["a"] = _padded(q)
        q, s["b_scale"] = _quantise(_values(c["b"], g, c["N"], c["K"]), c["b_block"])
        s["b"] = _padded(q)
        s["out"] = torch.empty(c["M"], c["N"], device="cuda", dtype=DTYPES[c["out"]])
    else:
        T, D = c["T"], c["D"]
        s["x"] = _randn(g, T, 4, D).to(BF16)
        # a memory that agrees a little with the first stream, so that the gates spread over (0, 1)
        s["k"] = _randn(g, T, D) + 2 / math.sqrt(D) * _randn(g, T, 1) * s["x"][:, 0].float()
        s["state"] = (_rand(g, T) < c["dead"]).to(torch.uint8)
        s["alpha"] = _randn(g, 4)
        s["dy"] = (_values("grad", g, T, 4 * D) * 10).reshape(T, 4, D).to(BF16)
        s["dx"] = torch.empty_like(s["x"])
        s["dk"] = torch.empty(T, D, device="cuda", dtype=DTYPES[c["dk"]])
        s["dalpha"] = torch.empty(4, device="cuda")
        s["workspace"] = torch.empty(1 << 20, device="cuda", dtype=torch.uint8)
    return s


# ------------------------------------------------------------------------ operators

EPS = 1e-6


def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _plain_embed(s):
    c, ids = s["case"], s["ids"].long()
    y = s["table"][ids.clamp(min=0)].float() * (ids >= 0).unsqueeze(-1)
    if c["pooled"]:
        y = y.sum(1)
    return (y * c["scale"]).to(DTYPES[c["out"]])


def _plain_grad(s):
    c, ids = s["case"], s["ids"].long()
    T, R, D = c["T"], c["R"], c["D"]
    dy = s["dy"].float()
    if c["pooled"]:
        dy = dy.unsqueeze(1).expand(T, R, D)
    dy = (dy * (ids >= 0).unsqueeze(-1)).reshape(T * R, D)
    if not c["sparse"]:
        grad = torch.zeros(c["rows"], D, device="cuda").index_add_(0, ids.reshape(-1).clamp(min=0), dy)
        return {"grad": (grad * c["scale"]).to(DTYPES[c["out"]])}
    key = torch.where(ids >= 0, ids, c["rows"]).reshape(-1)
    uniq, at = torch.unique(key, return_inverse=True)
    live = uniq < c["rows"]
    row_ids = torch.full((T * R,), -1, device="cuda", dtype=torch.int32)
    row_ids[:uniq.numel()] = torch.where(live, uniq, -1).to(torch.int32)
    grads = torch.zeros(T * R, D, device="cuda").index_add_(0, at, dy)
    return {"row_ids": row_ids, "grads": (grads * c["scale"]).to(DTYPES[c["out"]]),
            "count": live.sum().to(torch.int32).reshape(1)}


def _fp8_out(q, e, qt=None, et=None):
    out = {"q": q.view(torch.float8_e4m3fn), "s": e}
    if qt is not None:
        out |= {"qt": qt.view(torch.float8_e4m3fn), "st": et}
    return out


def _plain_quant(s):
    c, x = s["case"], s["x"].float()
    out = _quantise(x, c["block_rows"])
    if c["cols"]:
        out += _quantise(x.t().contiguous(), c["block_rows"])
    return _fp8_out(*out)


def _plain_matmul(s):
    c = s["case"]
    a = s["a"].contiguous().view(torch.float8_e4m3fn).float() * torch.exp2(_spread(s["a_scale"], 1, c["M"], c["K"]).float() - 127)
    b = s["b"].contiguous().view(torch.float8_e4m3fn).float() * torch.exp2(_spread(s["b_scale"], c["b_block"], c["N"], c["K"]).float() - 127)
    return (a @ b.t()).to(DTYPES[c["out"]])


def _plain_gate(s):
    c = s["case"]
    D = c["D"]
    live = (s["state"] == 0).unsqueeze(1)
    x0, k, dy, alpha = s["x"][:, 0].float(), s["k"] * live, s["dy"].float(), s["alpha"]
    ra = (x0.square().mean(1, keepdim=True) + EPS).rsqrt()
    rk = (k.square().mean(1, keepdim=True) + EPS).rsqrt()
    z = (x0 * k).sum(1, keepdim=True) * ra * rk / math.sqrt(D)
    gate = torch.sigmoid(z)
    by_stream = (dy * k.unsqueeze(1)).sum(2)  # <dy_s, k>
    dz = (by_stream * alpha).sum(1, keepdim=True) * gate * (1 - gate)
    common = ra * rk / math.sqrt(D)
    dx0 = dz * (common * k - z * ra * ra / D * x0) * live
    dk = gate * (dy * alpha.reshape(1, 4, 1)).sum(1) + dz * (common * x0 - z * rk * rk / D * k)
    dx = dy.clone()
    dx[:, 0] += dx0
    return {"dx": dx.to(BF16), "dk": (dk * live).to(DTYPES[c["dk"]]), "dalpha": (gate * live * by_stream).sum(0)}


_run_plain = {"embed": _plain_embed, "grad": _plain_grad, "quant": _plain_quant, "matmul": _plain_matmul,
              "gate": _plain_gate}


def _eg():
    import hashed_gram_memory_gb300
    return hashed_gram_memory_gb300


def _own_embed(s):
    c = s["case"]
    return _eg().engram_embed(s["ids"], s["table"], scale=c["scale"], pooled=c["pooled"], out=s["out"])


def _own_grad(s):
    c, eg = s["case"], _eg()
    if c["sparse"]:
        row_ids, grads, count = eg.engram_embed_grad_rows(
            s["ids"], s["dy"], c["rows"], scale=c["scale"], pooled=c["pooled"], row_ids=s["row_ids"],
            grads=s["grads"], count=s["count"], workspace=s["workspace"])
        return {"row_ids": row_ids, "grads": grads, "count": count}
    return {"grad": eg.engram_embed_grad(s["ids"], s["dy"], c["rows"], scale=c["scale"], pooled=c["pooled"],
                                         grad=s["grad"], workspace=s["workspace"])}


def _own_quant(s):
    c = s["case"]
    return _fp8_out(*_eg().engram_fp8_quantise(s["x"], block_rows=c["block_rows"], cols=c["cols"], out=s["q"]))


def _own_matmul(s):
    return _eg().engram_fp8_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], b_block=s["case"]["b_block"],
                                   out=s["out"])


def _own_gate(s):
    dx, dk, dalpha = _eg().engram_gate_add_grad(s["k"], s["state"], s["x"], s["alpha"], s["dy"], eps=EPS, dx=s["dx"],
                                                dk=s["dk"], dalpha=s["dalpha"], workspace=s["workspace"])
    return {"dx": dx, "dk": dk, "dalpha": dalpha}


_run_own = {"embed": _own_embed, "grad": _own_grad, "quant": _own_quant, "matmul": _own_matmul, "gate": _own_gate}


# --------------------------------------------------------------------------- exact

def _e4m3(v):
    """The nearest e4m3 value of each |v| <= 448, ties to even: a grid of 2^-9 below
    2^-6, of an eighth of the power of two above."""
    _, ex = torch.frexp(v)
    step = torch.exp2((ex.double() - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_quantise(x, br):
    """Block by block from the definition: 448 * 2^e is the first that reaches the largest
    magnitude."""
    M, K = x.shape
    out = torch.empty_like(x)
    for k0 in range(0, K, 128):
        part = x[:, k0:k0 + 128]
        big = part.abs().amax(1)
        if br > 1:
            big = torch.stack([b.amax() for b in big.split(br)]).repeat_interleave(br)[:M]
        e = torch.ceil(torch.log2(big / 448)).clamp(min=-127)
        e = e + (torch.exp2(e) * 448 < big) - (torch.exp2(e - 1) * 448 >= big).double() * (e > -127)
        out[:, k0:k0 + 128] = _e4m3(part * torch.exp2(-e).unsqueeze(1))
    return out


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    f8 = torch.float64
    if op == "embed":
        out = torch.empty(s["out"].shape, device="cuda", dtype=f8)
        padded = torch.cat([s["table"], torch.zeros(1, c["D"], device="cuda", dtype=s["table"].dtype)])
        for t in range(0, c["T"], 4096):
            rows = padded[s["ids"][t:t + 4096].long()].to(f8) * c["scale"]  # -1 is the row of zeros
            out[t:t + 4096] = rows.sum(1) if c["pooled"] else rows
        return out
    if op == "grad":
        T, R, D = c["T"], c["R"], c["D"]
        flat = s["ids"].reshape(-1).long()
        order = torch.argsort(flat, stable=True)
        order = order[int((flat < 0).sum()):]
        ids, runs = torch.unique_consecutive(flat[order], return_counts=True)
        src = order // R if c["pooled"] else order
        dy = s["dy"].reshape(-1, D)
        n = ids.numel()
        grads = torch.zeros(T * R if c["sparse"] else c["rows"], D, device="cuda", dtype=f8)
        seg = torch.repeat_interleave(torch.arange(n, device="cuda") if c["sparse"] else ids, runs)
        for i in range(0, src.numel(), 1 << 18):
            grads.index_add_(0, seg[i:i + (1 << 18)], dy[src[i:i + (1 << 18)]].to(f8))
        grads *= c["scale"]
        return {"row_ids": None, "grads": grads, "count": None} if c["sparse"] else {"grad": grads}
    if op == "quant":
        x = s["x"].to(f8)
        out = {"q": _exact_quantise(x, c["block_rows"]), "s": None}
        if c["cols"]:
            out |= {"qt": _exact_quantise(x.t().contiguous(), c["block_rows"]), "st": None}
        return out
    if op == "matmul":
        out = torch.zeros(c["M"], c["N"], device="cuda", dtype=f8)
        for kb in range(0, c["K"], 2048):
            part = []
            for q, e, br in ((s["a"], s["a_scale"], 1), (s["b"], s["b_scale"], c["b_block"])):
                v = q[:, kb:kb + 2048].contiguous().view(torch.float8_e4m3fn).to(f8)
                w = torch.pow(2.0, e[:, kb // 128:kb // 128 + 16].to(f8) - 127)
                w = w.repeat_interleave(128, 1)[:, :v.shape[1]]
                part.append(v * (w.repeat_interleave(br, 0)[:v.shape[0]] if br > 1 else w))
            out.addmm_(part[0], part[1].t())
        return out
    T, D = c["T"], c["D"]
    dx = torch.empty(T, 4, D, device="cuda", dtype=f8)
    dk = torch.empty(T, D, device="cuda", dtype=f8)
    dalpha = torch.zeros(4, device="cuda", dtype=f8)
    alpha = s["alpha"].to(f8)
    for t in range(0, T, 8192):
        at = slice(t, t + 8192)
        live = (s["state"][at] == 0).to(f8)
        a, k, dy = s["x"][at, 0].to(f8), s["k"][at].to(f8), s["dy"][at].to(f8)
        na = (a.pow(2).sum(1) / D + EPS).sqrt()
        nk = (k.pow(2).sum(1) / D + EPS).sqrt()
        ua, uk = a / na[:, None], k / nk[:, None]  # the normalised vectors
        z = (ua * uk).sum(1) / math.sqrt(D)
        gate = 1 / (1 + torch.exp(-z))
        c_vec = torch.einsum("tsd,s->td", dy, alpha)
        dot = torch.einsum("tsd,td->ts", dy, k)
        dz = (c_vec * k).sum(1) * gate * (1 - gate) / math.sqrt(D) * live
        # through u = v / n: dv = (du - u <u, du> / D) / n
        da = (uk - ua * ((ua * uk).sum(1) / D)[:, None]) / na[:, None] * dz[:, None]
        dku = (ua - uk * ((ua * uk).sum(1) / D)[:, None]) / nk[:, None] * dz[:, None]
        dx[at] = dy
        dx[at, 0] += da
        dk[at] = (gate[:, None] * c_vec) * live[:, None] + dku
        dalpha += (dot * (gate * live)[:, None]).sum(0)
    return {"dx": dx, "dk": dk, "dalpha": dalpha}
