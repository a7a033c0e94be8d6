"""Trains one transformer block with the library's operators between its
matrix products, keeping what its backward pass needs in 8 bits.

The model is an embedding, one pre-norm block (causal attention with rotary
positions and grouped keys, a gated activation) and an output matrix, over one
flat bf16 parameter buffer with fp32 master weights (the layout
mp_optimizer_step takes). Per step, the products and the attention's softmax
being PyTorch's:

  x = the tokens' embeddings
  y = RMS norm of x; x kept in 8 bits                  mp_rmsnorm_forward
  q, k turned by their positions                       mp_rope
  h = x + attention; z = RMS norm of h; h in 8 bits    mp_rmsnorm_forward
  a = silu(gate) * up; gate and up in 8 bits           mp_gated_forward
  logits = RMS norm of (h + a W) times O               mp_rmsnorm_forward
  log p(next token), gradient of the logits            mp_token_logprob_forward, _backward
  the same backwards, from the 8 bits                  mp_rmsnorm_backward, mp_gated_backward,
                                                       mp_rope (inverse)
  norm, clipping, AdamW, stochastic rounding           mp_optimizer_step

  python examples/train_block.py [--steps N] [--seed S]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_adamw_gb300 as mp  # noqa: E402

EPS = 1e-5


class Block:
    """Embedding, one block and output matrix in one flat buffer."""

    def __init__(self, vocab=1003, width=256, heads=4, kv_heads=2, inner=512, batch=4, length=64, lr=2e-3, seed=0,
                 dtype=torch.bfloat16):
        self.vocab, self.width, self.heads, self.kv_heads, self.inner = vocab, width, heads, kv_heads, inner
        self.batch, self.length, self.dim, self.dtype = batch, length, width // heads, dtype
        qkv = (heads + 2 * kv_heads) * self.dim
        self.shapes = {"embedding": (vocab, width), "norm1": (width,), "wqkv": (qkv, width), "wo": (width, width),
                       "norm2": (width,), "gate_up": (2 * inner, width), "down": (width, inner), "norm3": (width,),
                       "output": (vocab, width)}
        table, views, at = [], {}, 0
        for name, shape in self.shapes.items():
            n = math.prod(shape)
            table.append((at, n, int(len(shape) == 2)))
            views[name] = (at, n, shape)
            at += n
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.master = torch.empty(at, device="cuda").normal_(0.0, 0.02, generator=gen)
        for name, (o, n, shape) in views.items():
            if len(shape) == 1:
                self.master[o:o + n] = 1.0
        self.params = self.master.to(dtype)
        self.grads = torch.zeros_like(self.params)
        self.m, self.v = torch.zeros_like(self.master), torch.zeros_like(self.master)
        self.p = {k: self.params[o:o + n].view(s) for k, (o, n, s) in views.items()}
        self.g = {k: self.grads[o:o + n].view(s) for k, (o, n, s) in views.items()}
        self.opt = mp.Optimizer(table, lr=lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.01, clip=1.0)
        self.t = 0
        rows = batch * length
        self.positions = torch.arange(length, device="cuda").repeat(batch)
        self.turns, self.factor = mp.mp_rope_frequencies(self.dim)
        self.mask = torch.ones(length, length, dtype=torch.bool, device="cuda").tril()

        def new(*shape):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        def new8(d):
            return (torch.empty(rows, d, dtype=torch.uint8, device="cuda"),
                    torch.empty(rows, -(-d // 32), dtype=torch.uint8, device="cuda"))
        self.y = [new(rows, width) for _ in range(3)]
        self.h = [None] + [new(rows, width) for _ in range(2)]
        self.rstd = [torch.empty(rows, device="cuda") for _ in range(3)]
        self.h8 = [new8(width) for _ in range(3)]
        self.q, self.k = new(rows, heads, self.dim), new(rows, kv_heads, self.dim)
        self.act, self.gate8, self.up8 = new(rows, inner), new8(inner), new8(inner)
        self.workspace = torch.empty(mp.mp_rmsnorm_workspace_bytes(rows, width), dtype=torch.uint8, device="cuda")

    def norm(self, i, x, residual=None):
        name = f"norm{i + 1}"
        mp.mp_rmsnorm_forward(self.y[i], x, self.p[name], EPS, residual=residual, h=self.h[i], rstd=self.rstd[i],
                              h8=self.h8[i][0], h8_scale=self.h8[i][1])
        return self.y[i]

    def norm_back(self, i, dy, dh=None):
        name = f"norm{i + 1}"
        dx = torch.empty_like(dy)
        mp.mp_rmsnorm_backward(dx, self.g[name], dy, self.h8[i][0], self.p[name], self.rstd[i], dh=dh,
                               h_scale=self.h8[i][1], workspace=self.workspace)
        return dx

    def _by_head(self, x, heads):
        """[rows, heads, dim] -> [batch, heads, length, dim], keys and values once for each query head."""
        x = x.view(self.batch, self.length, heads, self.dim).transpose(1, 2)
        return x.repeat_interleave(self.heads // heads, 1).float()

    def _by_row(self, x, heads):
        x = x.view(self.batch, heads, self.heads // heads, self.length, self.dim).sum(2)
        return x.transpose(1, 2).reshape(-1, heads, self.dim).to(self.dtype)

    def forward(self, tokens):
        """Logits of [batch, length] tokens."""
        H, K, D = self.heads, self.kv_heads, self.dim
        x = self.p["embedding"][tokens.view(-1)]
        qkv = self.norm(0, x) @ self.p["wqkv"].t()
        parts = qkv.view(-1, H + 2 * K, D).split((H, K, K), 1)
        mp.mp_rope(self.q, parts[0], self.k, parts[1], self.turns, self.positions, factor=self.factor)
        q, k, self.value = self._by_head(self.q, H), self._by_head(self.k, K), self._by_head(parts[2], K)
        scores = (q @ k.transpose(2, 3) * D ** -0.5).masked_fill(~self.mask, -math.inf)
        self.prob = torch.softmax(scores, 3)
        self.mixed = self._by_row((self.prob @ self.value).contiguous(), H).view(-1, self.width)
        z = self.norm(1, self.mixed @ self.p["wo"].t(), x)
        both = z @ self.p["gate_up"].t()
        mp.mp_gated_forward(self.act, both[:, :self.inner], both[:, self.inner:], gate8=self.gate8[0],
                            gate8_scale=self.gate8[1], up8=self.up8[0], up8_scale=self.up8[1])
        return self.norm(2, self.act @ self.p["down"].t(), self.h[1]) @ self.p["output"].t()

    def backward(self, tokens, d_logits):
        """The gradients of all parameters, into the flat buffer."""
        H, K, D, g = self.heads, self.kv_heads, self.dim, self.g
        torch.matmul(d_logits.t(), self.y[2], out=g["output"])
        d_h = self.norm_back(2, d_logits @ self.p["output"])  # of h + a W: of both
        d_act = d_h @ self.p["down"]
        d_both = torch.empty(d_h.shape[0], 2 * self.inner, dtype=self.dtype, device="cuda")
        mp.mp_gated_backward(d_both[:, :self.inner], d_both[:, self.inner:], d_act, self.gate8[0], self.up8[0],
                             gate_scale=self.gate8[1], up_scale=self.up8[1], y=self.act)
        torch.matmul(d_h.t(), self.act, out=g["down"])
        torch.matmul(d_both.t(), self.y[1], out=g["gate_up"])
        d_h = self.norm_back(1, d_both @ self.p["gate_up"], d_h)
        torch.matmul(d_h.t(), self.mixed, out=g["wo"])
        d_mixed = self._by_head((d_h @ self.p["wo"]).view(-1, H, D), H)
        d_value = self.prob.transpose(2, 3) @ d_mixed
        d_prob = d_mixed @ self.value.transpose(2, 3)
        d_scores = self.prob * (d_prob - (d_prob * self.prob).sum(3, keepdim=True)) * D ** -0.5
        d_q = self._by_row((d_scores @ self._by_head(self.k, K)).contiguous(), H)
        d_k = self._by_row((d_scores.transpose(2, 3) @ self._by_head(self.q, H)).contiguous(), K)
        mp.mp_rope(d_q, d_q, d_k, d_k, self.turns, self.positions, inverse=True, factor=self.factor)
        d_qkv = torch.cat((d_q, d_k, self._by_row(d_value.contiguous(), K)), 1).view(-1, (H + 2 * K) * D)
        torch.matmul(d_qkv.t(), self.y[0], out=g["wqkv"])
        d_x = self.norm_back(0, d_qkv @ self.p["wqkv"], d_h)
        g["embedding"].copy_(torch.zeros(self.shapes["embedding"], device="cuda").index_add_(0, tokens.view(-1),
                                                                                             d_x.float()))

    def step(self):
        self.t += 1
        self.opt.step(self.params, self.grads, self.master, self.m, self.v, t=self.t, seed=self.t)


def train(steps=200, seed=0):
    """Mean losses over the first and the last hundredth of the steps."""
    model = Block(seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    follow = torch.randint(0, model.vocab, (model.vocab, 4), generator=gen, device="cuda")  # a token's likely successors
    rows = model.batch * model.length
    logp, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    d_logp = torch.full((rows,), -1.0 / rows, device="cuda")  # loss = mean of -log p
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    losses = []
    for _ in range(steps):
        text = torch.randint(0, model.vocab, (model.batch, model.length + 1), generator=gen, device="cuda")
        pick = torch.randint(0, 4, text.shape, generator=gen, device="cuda")
        for i in range(1, model.length + 1):
            text[:, i] = follow[text[:, i - 1], pick[:, i]]
        tokens, target = text[:, :-1].contiguous(), text[:, 1:].reshape(-1)
        logits = model.forward(tokens)
        mp.mp_token_logprob_forward(logits, target, logp=logp, lse=lse, d_status=status)
        losses.append(-logp.mean())
        mp.mp_token_logprob_backward(logits, logits, target, lse=lse, dlogp=d_logp)  # over the logits
        model.backward(tokens, logits)
        model.step()
    model.opt.check_status()
    if int(status):
        raise mp.MpError(int(status), "train_block")
    losses = torch.stack(losses)
    k = max(1, steps // 100)
    return float(losses[:k].mean()), float(losses[-k:].mean())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    print("cross entropy: %.3f -> %.3f" % train(a.steps, a.seed))


if __name__ == "__main__":
    main()
