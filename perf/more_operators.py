"""The bf16 product with an epilogue, its gradient and the orthogonalised update, case by case.

Three operators, each called as a training or serving program calls it:

  matmul  engram_matmul         act(scale * a b^T + bias) + residual, keeping the pre-activation if asked
  grad    engram_matmul_grad    its backward pass: the gradients of a, b and the bias
  orth    engram_orthogonalise  a momentum step and the Newton-Schulz iteration on it (an optimiser's
                                orthogonal update of a weight matrix)

`run` calls them where `own` is true; elsewhere it computes the same in elementary
torch operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

HIDDEN = 4096    # hidden size of the streams
CONCAT = 6144    # a token's 3 x 8 rows of 256, concatenated
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}
BYTES = {"bf16": 2, "f32": 4, "": 0}
STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
BETA = 0.95
EPS = 1e-7


# --------------------------------------------------------------------------- cases

def _matmul(name, M, N, K, out, act="none", bias=True, residual="", pre="", b="nk", pad=0):
    """residual, pre: their type, or "" for none.  b: the weights' layout in memory.  pad:
    columns between the rows of a."""
    return {"name": name, "op": "matmul", "M": M, "N": N, "K": K, "out": out, "act": act, "bias": bias,
            "residual": residual, "pre": pre, "b": b, "pad": pad}


def _grad(name, M, N, K, dy, da, db, act="none", pre="", dbias=True, accumulate=False):
    return {"name": name, "op": "grad", "M": M, "N": N, "K": K, "dy": dy, "da": da, "db": db, "act": act,
            "pre": pre, "dbias": dbias, "accumulate": accumulate}


def _orth(name, L, M, N, g, momentum=True, nesterov=True):
    return {"name": name, "op": "orth", "L": L, "M": M, "N": N, "g": g, "momentum": momentum,
            "nesterov": nesterov}


def listed():
    return [
        # the connection's projection for one new token, and for a few decode slots with the
        # activation and the residual of a serving block
        _matmul("matmul_one_token", 1, HIDDEN, CONCAT, "f32"),
        _matmul("matmul_decode", 37, HIDDEN, CONCAT, "bf16", act="silu", residual="bf16"),
        # odd sizes whose rows do not start on 16 bytes, weights stored the other way round
        _matmul("matmul_ragged", 1003, 1278, 475, "bf16", act="gelu", pre="bf16", b="kn"),
        # the projection of a full prefill with its bias and residual
        _matmul("matmul_prefill", 65536, HIDDEN, CONCAT, "bf16", residual="bf16"),
        # a unit test's size: rows of 2 heads x 256, every gradient
        _grad("grad_tiny", 256, 256, 1536, "bf16", "bf16", "bf16", act="relu", pre="bf16"),
        # a step over 512 slots through an activation
        _grad("grad_512", 512, HIDDEN, CONCAT, "bf16", "bf16", "bf16", act="gelu", pre="bf16"),
        # a ragged batch of tokens into odd widths
        _grad("grad_ragged", 16411, 2573, 1278, "f32", "bf16", "bf16", act="silu", pre="f32"),
        # a 16k-token step: the weight gradient added to the fp32 one of the step before
        _grad("grad_16k", 16384, HIDDEN, CONCAT, "bf16", "bf16", "f32", accumulate=True),
        # updates of the tiny connection's matrix, of a tall one with odd sides, of the same
        # matrix of several layers at once, and of the connection's projection
        _orth("orth_tiny", 1, 256, 1536, "f32"),
        _orth("orth_tall", 1, 5888, 475, "bf16", nesterov=False),
        _orth("orth_layers", 12, 1024, 1536, "bf16"),
        _orth("orth_projection", 1, HIDDEN, CONCAT, "f32"),
    ]


LARGEST = 2 * 65536 * HIDDEN * CONCAT  # operations of the largest listed case


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step=64):
    """A width in [lo, hi]: mostly a multiple of `step`, sometimes any."""
    w = _log(rng, lo, hi)
    return max(step, w // step * step) if rng.random() < 0.6 else w


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul", "grad", "grad", "orth", "orth"])
    if op == "orth":
        M, N = _width(rng, 16, 6144), _width(rng, 16, 6144)
        r, c = min(M, N), max(M, N)
        L = _log(rng, 1, max(1, min(32, LARGEST // 4 // (STEPS * (4 * r * r * c + 2 * r ** 3)))))
        momentum = rng.random() < 0.7
        c = _orth("", L, M, N, rng.choice(["bf16", "f32"]), momentum, momentum and rng.random() < 0.6)
    else:
        N, K = _width(rng, 16, 8192), _width(rng, 16, 8192)
        M = _log(rng, 1, max(1, min(65536, LARGEST // 2 // (N * K) // (1 if op == "matmul" else 4))))
        act = rng.choice(["none", "none", "relu", "silu", "gelu"])
        if op == "matmul":
            c = _matmul("", M, N, K, rng.choice(["bf16", "f32"]), act, rng.random() < 0.7,
                        rng.choice(["", "", "bf16", "f32"]), rng.choice(["", "", "bf16", "f32"]),
                        rng.choice(["nk", "nk", "kn"]), rng.choice([0, 0, 8, 3]))
        else:
            # through an activation, or from an fp32 gradient, what the products read has 8 bits
            dy = rng.choice(["bf16", "f32"])
            exactly = act == "none" and dy == "bf16"
            c = _grad("", M, N, K, dy, "bf16", rng.choice(["bf16", "f32"]) if exactly else "bf16", act,
                      "" if act == "none" else rng.choice(["bf16", "f32"]), rng.random() < 0.7,
                      rng.random() < 0.3)
    del c["name"]
    return c


def work(c):
    if c["op"] == "orth":
        n, r, w = c["L"] * c["M"] * c["N"], min(c["M"], c["N"]), max(c["M"], c["N"])
        # the two symmetric products are needed on one side of their diagonal
        return {"bytes": n * (BYTES[c["g"]] + (8 if c["momentum"] else 0) + 2),
                "flops": c["L"] * STEPS * (3 * r * r * w + r ** 3)}
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] == "matmul":
        return {"bytes": 2 * (M + N) * K + M * N * (BYTES[c["out"]] + BYTES[c["residual"]] + BYTES[c["pre"]])
                + (4 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    more = 2 if c["accumulate"] else 1
    return {"bytes": 2 * (M + N) * K + M * N * (BYTES[c["dy"]] + BYTES[c["pre"]]) + M * K * BYTES[c["da"]]
            + N * K * BYTES[c["db"]] * more + (4 * N * more if c["dbias"] else 0), "flops": 4 * M * N * K}


# -------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _empty(dtype, *shape):
    return torch.empty(*shape, device="cuda", dtype=DTYPES[dtype])


def _prepare_matmul(c, g, s):
    M, N, K = c["M"], c["N"], c["K"]
    s["a"] = _randn(g, M, K + c["pad"]).to(BF16)[:, :K]
    w = _randn(g, N, K) if c["b"] == "nk" else _randn(g, K, N)
    w = (w / math.sqrt(K)).to(BF16)
    s["b"] = w if c["b"] == "nk" else w.t()
    s["bias"] = 0.5 * _randn(g, N) if c["bias"] else None
    s["residual"] = _randn(g, M, N).to(DTYPES[c["residual"]]) if c["residual"] else None
    s["pre"] = _empty(c["pre"], M, N) if c["pre"] else None
    s["out"] = _empty(c["out"], M, N)


def _prepare_grad(c, g, s):
    M, N, K = c["M"], c["N"], c["K"]
    s["a"] = _randn(g, M, K).to(BF16)
    s["b"] = (_randn(g, N, K) / math.sqrt(K)).to(BF16)
    # a size of its own for each token, and a mean, as a bias meets
    dy = _randn(g, M, N) + 0.1 * _randn(g, N)
    s["dy"] = (1e-3 * torch.exp(_randn(g, M, 1)) * dy).to(DTYPES[c["dy"]])
    s["pre"] = _randn(g, M, N).to(DTYPES[c["pre"]]) if c["pre"] else None
    s["da"] = _empty(c["da"], M, K)
    s["db"], s["dbias"] = _empty(c["db"], N, K), _empty("f32", N) if c["dbias"] else None
    if c["accumulate"]:
        s["db"].copy_(_randn(g, N, K) * 1e-2)
        if c["dbias"]:
            s["dbias"].copy_(_randn(g, N) * 1e-2)


def _prepare_orth(c, g, s):
    L, M, N = c["L"], c["M"], c["N"]
    # a batch's gradient: noise with a size for each row, and a few directions that stand out
    low = _randn(g, L, M, 4) @ _randn(g, L, 4, N)
    s["g"] = (1e-3 * (_randn(g, L, M, N) * torch.exp(0.5 * _randn(g, L, M, 1)) + low)).to(DTYPES[c["g"]])
    s["momentum"] = 3e-3 * _randn(g, L, M, N) if c["momentum"] else None
    s["out"] = _empty("bf16", L, M, N)


def prepare(case, seed):
    s = {"case": case}
    {"matmul": _prepare_matmul, "grad": _prepare_grad, "orth": _prepare_orth}[case["op"]](case, _gen(seed), s)
    return s


# ------------------------------------------------------------------------ operators

def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))


def _plain_matmul(s):
    c = s["case"]
    z = s["a"].float() @ s["b"].float().t()
    if c["bias"]:
        z = z + s["bias"]
    y = _act(z, c["act"])
    if c["residual"]:
        y = y + s["residual"].float()
    return {"out": y.to(DTYPES[c["out"]]), "pre": z.to(DTYPES[c["pre"]]) if c["pre"] else None}


def _plain_grad(s):
    c = s["case"]
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(s["pre"].float(), c["act"])
    db, dbias = dz.t() @ s["a"].float(), dz.sum(0)
    if c["accumulate"]:
        db, dbias = s["db"].copy_(db + s["db"].float()), s["dbias"].add_(dbias) if c["dbias"] else None
    return {"da": (dz @ s["b"].float()).to(DTYPES[c["da"]]), "db": db.to(DTYPES[c["db"]]),
            "dbias": dbias if c["dbias"] else None}


def _plain_orth(s):
    c, u = s["case"], s["g"].float()
    m = s["momentum"]
    if m is not None:
        m.mul_(BETA).add_(u)
        u = u + BETA * m if c["nesterov"] else m
    x = u / (u.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    if c["M"] > c["N"]:
        x = x.transpose(1, 2)
    a, b, d = COEFFICIENTS
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + d * (gram @ gram)) @ x
    if c["M"] > c["N"]:
        x = x.transpose(1, 2)
    return {"out": x.to(BF16).contiguous(), "momentum": m}


_run_plain = {"matmul": _plain_matmul, "grad": _plain_grad, "orth": _plain_orth}


def _eg():
    import hashed_gram_memory_gb300
    return hashed_gram_memory_gb300


def _own_act(c):
    return getattr(_eg(), "ACT_" + c["act"].upper())


def _own_matmul(s):
    c = s["case"]
    out = _eg().engram_matmul(s["a"], s["b"], bias=s["bias"], activation=_own_act(c), residual=s["residual"],
                              pre=s["pre"], out=s["out"])
    return {"out": out, "pre": s["pre"]}


def _own_grad(s):
    c = s["case"]
    da, db, dbias = _eg().engram_matmul_grad(s["dy"], s["a"], s["b"], pre=s["pre"], activation=_own_act(c),
                                             grad_bias=c["dbias"], accumulate=c["accumulate"], da=s["da"],
                                             db=s["db"], dbias=s["dbias"])
    return {"da": da, "db": db, "dbias": dbias}


def _own_orth(s):
    c = s["case"]
    out = _eg().engram_orthogonalise(s["g"], momentum=s["momentum"], beta=BETA, nesterov=c["nesterov"],
                                     steps=STEPS, coefficients=COEFFICIENTS, eps=EPS, out=s["out"])
    return {"out": out, "momentum": s["momentum"]}


_run_own = {"matmul": _own_matmul, "grad": _own_grad, "orth": _own_orth}


# --------------------------------------------------------------------------- exact

def _phi(z):
    """The normal distribution below z."""
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def exact(case, seed):
    c, f8 = case, torch.float64
    s = prepare(case, seed)
    if c["op"] == "matmul":
        wide, b = torch.empty(c["M"], c["N"], device="cuda", dtype=f8), s["b"].to(f8)
        out, pre = wide, torch.empty_like(wide) if c["pre"] else None
        for m in range(0, c["M"], 8192):
            at = slice(m, m + 8192)
            z = torch.einsum("mk,nk->mn", s["a"][at].to(f8), b)
            if c["bias"]:
                z += s["bias"].to(f8)[None]
            if c["pre"]:
                pre[at] = z
            y = {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, torch.zeros_like(z)),
                 "silu": lambda: z * torch.sigmoid(z), "gelu": lambda: z * _phi(z)}[c["act"]]()
            out[at] = y + s["residual"][at].to(f8) if c["residual"] else y
        return {"out": out, "pre": pre}
    if c["op"] == "grad":
        db, dbias = torch.zeros(c["N"], c["K"], device="cuda", dtype=f8), torch.zeros(c["N"], device="cuda", dtype=f8)
        if c["accumulate"]:
            db += s["db"]
            if c["dbias"]:
                dbias += s["dbias"]
        da, b = torch.empty(c["M"], c["K"], device="cuda", dtype=f8), s["b"].to(f8)
        for m in range(0, c["M"], 8192):
            at = slice(m, m + 8192)
            dz, a = s["dy"][at].to(f8), s["a"][at].to(f8)
            if c["act"] != "none":
                z = s["pre"][at].to(f8)
                p = torch.sigmoid(z)
                dz = dz * {"relu": lambda: torch.sign(z).clamp(min=0), "silu": lambda: p + z * p - z * p * p,
                           "gelu": lambda: _phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)}[c["act"]]()
            da[at] = torch.einsum("mn,nk->mk", dz, b)
            db += torch.einsum("mn,mk->nk", dz, a)
            dbias += torch.einsum("mn->n", dz)
        return {"da": da, "db": db, "dbias": dbias if c["dbias"] else None}
    out, a, b, d = [], *COEFFICIENTS
    moved = torch.empty(c["L"], c["M"], c["N"], device="cuda", dtype=f8) if c["momentum"] else None
    for i in range(c["L"]):
        u = s["g"][i].to(f8)
        if c["momentum"]:
            moved[i] = s["momentum"][i].to(f8) * BETA + u
            u = u + moved[i] * BETA if c["nesterov"] else moved[i]
        x = u / (torch.sqrt(torch.einsum("mn,mn->", u, u)) + EPS)
        for _ in range(STEPS):  # a x + b x x'x + d x x'x x'x
            inner = x.t() @ x if c["M"] > c["N"] else x @ x.t()
            power = inner @ inner
            x = a * x + (x @ inner * b + x @ power * d if c["M"] > c["N"] else inner @ x * b + power @ x * d)
        out.append(x)
    return {"out": torch.stack(out), "momentum": moved}
