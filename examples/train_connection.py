"""Training steps of the Engram connection: the hashed table, the wkv matrix and alpha
learn to carry the streams to given targets.

Forward, per step: ids are hashed into row ids, their rows looked up and concatenated
(engram_embed), quantised to e4m3 with a scale per block of 128 and multiplied by wkv in
the same form (engram_fp8_quantise, engram_fp8_matmul), gated and added into the streams
(engram_gate_add).  Backward: the gate's gradients (engram_gate_add_grad), the two 8-bit
products of the projection's backward pass, and the gradient of the rows that the tokens
named (engram_embed_grad_rows), which is all of the table that a step touches.

The quantiser's transposed copies make every product a row-times-row one: E and dk are
each read once for both of theirs.

  python examples/train_connection.py [--tokens 4096] [--steps 30]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hashed_gram_memory_gb300 as eg  # noqa: E402


class Connection:
    """A table of hashed rows (bf16 [rows, d]) shared by the three n-gram orders, cut into
    prime buckets, and the projection to `hidden` columns (fp32, quantised each step)."""

    def __init__(self, n_eids=1000, heads=2, d=64, hidden=256, hash_vocab=500, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.d, self.hidden, self.n_eids = heads, d, hidden, n_eids
        self.primes = eg.engram_bucket_primes(1, 4, heads, hash_vocab)[0]
        self.rows = sum(sum(p) for p in self.primes)
        self.K = 3 * heads * d
        self.table = (torch.randn(self.rows, d, generator=g, device="cuda") * 0.02).bfloat16()
        self.wkv = torch.randn(hidden, self.K, generator=g, device="cuda")
        self.alpha = torch.full((4,), 0.5, device="cuda")
        self.tid2eid = torch.arange(1, n_eids + 1, device="cuda", dtype=torch.int32)
        self.status = torch.zeros(1, device="cuda", dtype=torch.int32)

    def row_ids(self, tokens, dead=None):
        """int32 [tokens, 3 * heads] for token ids [batch, seq] (dead tokens: all -1)."""
        ids = eg.engram_compress_hash(tokens, self.tid2eid, self.n_eids, self.heads, None, dead=dead,
                                      primes=self.primes, status=self.status)
        return ids.view(-1, 3 * self.heads)

    def forward(self, ids, x):
        """The streams x bf16 [tokens, 4, hidden] with the gated memory added, and what the
        backward pass needs."""
        T = ids.shape[0]
        e = eg.engram_embed(ids, self.table, status=self.status).view(T, self.K)
        q, s, qt, st = eg.engram_fp8_quantise(e, cols=True, status=self.status)
        w = eg.engram_fp8_quantise(self.wkv, block_rows=eg.FP8_BLOCK, cols=True, status=self.status)
        k = eg.engram_fp8_matmul(q, s, w[0], w[1], b_block=eg.FP8_BLOCK, status=self.status)
        state = (ids[:, 0] < 0).to(torch.uint8)
        y = eg.engram_gate_add(k, state, x, self.alpha)
        return y, (ids, x, k, state, (qt, st), w)

    def backward(self, saved, dy):
        """dx, dalpha, dwkv, and the table's gradient as (row ids, rows, count)."""
        ids, x, k, state, (qt, st), w = saved
        T = ids.shape[0]
        dx, dk, dalpha = eg.engram_gate_add_grad(k, state, x, self.alpha, dy)
        q, s, kt, ks = eg.engram_fp8_quantise(dk, cols=True, status=self.status)
        de = eg.engram_fp8_matmul(q, s, w[2], w[3], b_block=eg.FP8_BLOCK, out_dtype=torch.bfloat16,
                                  status=self.status)
        dwkv = eg.engram_fp8_matmul(kt, ks, qt, st, status=self.status)
        rows = eg.engram_embed_grad_rows(ids, de.view(T, -1, self.d), self.rows, status=self.status)
        return dx, dalpha, dwkv, rows

    def update(self, dalpha, dwkv, rows, lr):
        """A step against each gradient, scaled to unit root mean square, and on the table's
        touched rows alone; lr: the steps of the table, wkv and alpha."""
        row_ids, grads, count = rows
        n = int(count)
        at = row_ids[:n].long()

        def step(g, size):
            return g * (size / (g.square().mean().sqrt() + 1e-12))
        self.table[at] = (self.table[at].float() - step(grads[:n], lr[0])).bfloat16()
        self.wkv -= step(dwkv, lr[1])
        self.alpha -= step(dalpha, lr[2])


def train(tokens=4096, steps=30, lr=(0.005, 0.02, 0.02), seed=0):
    """Mean squared errors before each step."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    net = Connection(seed=seed)
    ids = torch.randint(0, net.n_eids, (1, tokens), generator=g, device="cuda", dtype=torch.int32)
    dead = (torch.rand(1, tokens, generator=g, device="cuda") < 0.05).to(torch.uint8)
    x = torch.randn(tokens, 4, net.hidden, generator=g, device="cuda").bfloat16()
    # a target that the memory can learn: a shift per token id in every stream
    shift = torch.randn(net.n_eids, 1, net.hidden, generator=g, device="cuda")
    target = x.float() + shift[ids.view(-1).long()]
    rows = net.row_ids(ids, dead)
    losses = []
    for _ in range(steps):
        y, saved = net.forward(rows, x)
        err = y.float() - target
        losses.append(float(err.square().mean()))
        _, dalpha, dwkv, grad = net.backward(saved, (err * (2 / tokens)).bfloat16())
        net.update(dalpha, dwkv, grad, lr)
    code, flags = eg.engram_read_status(net.status)
    if code != eg.OK:
        raise RuntimeError(f"status {flags:#x}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.tokens, a.steps)):
        print(f"step {i}: mean squared error {loss:.5f}")
