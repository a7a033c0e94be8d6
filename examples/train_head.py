"""Trains a small language model's head with the library's operators, then
distils it into a smaller one.

The model is an embedding, a layer norm and an output matrix, over one flat
bf16 parameter buffer with fp32 master weights (the
layout mp_optimizer_step takes). Per step:

  y = layer norm of the tokens' embeddings          mp_layernorm_forward
  logits = y O^T                                    (a plain matrix product)
  log p(next token)                                 mp_token_logprob_forward
  gradient of the logits                            mp_token_logprob_backward
  gradient of y, O                                  (plain matrix products)
  gradient of the embeddings, weight and bias       mp_layernorm_backward
  norm, clipping, AdamW, stochastic rounding        mp_optimizer_step

The teacher's 16 top alternatives (mp_token_logprob_forward's top_logp and
top_index) are then all the smaller model sees of it: mp_distill_topk gives the
loss and the gradient of its logits, and the rest of the step is the same.

  python examples/train_head.py [--steps N] [--seed S]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_adamw_gb300 as mp  # noqa: E402

EPS = 1e-5


class Head:
    """Embedding, layer norm and output matrix in one flat buffer."""

    def __init__(self, vocab, width, rows, lr, seed):
        self.vocab, self.width = vocab, width
        sizes = [vocab * width, width, width, vocab * width]
        offsets = [sum(sizes[:i]) for i in range(4)]
        table = [(o, n, int(n > width)) for o, n in zip(offsets, sizes)]
        n = sum(sizes)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.master = torch.zeros(n, device="cuda")
        self.master[:sizes[0]].normal_(0.0, 0.02, generator=gen)
        self.master[offsets[3]:].normal_(0.0, 0.02, generator=gen)
        self.master[offsets[1]:offsets[2]] = 1.0
        self.params = self.master.to(torch.bfloat16)
        self.grads = torch.zeros_like(self.params)
        self.m, self.v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        self.opt = mp.Optimizer(table, lr=lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.01, clip=1.0)
        self.t = 0

        def views(flat):
            e, w, b, out = (flat[o:o + k] for o, k in zip(offsets, sizes))
            return e.view(vocab, width), w, b, out.view(vocab, width)
        self.embedding, self.weight, self.bias, self.output = views(self.params)
        self.d_embedding, self.d_weight, self.d_bias, self.d_output = views(self.grads)
        bf, f = dict(dtype=torch.bfloat16, device="cuda"), dict(device="cuda")
        self.y, self.mean, self.rstd = torch.empty(rows, width, **bf), torch.empty(rows, **f), torch.empty(rows, **f)
        self.d_x = torch.empty(rows, width, **bf)
        self.workspace = torch.empty(mp.mp_layernorm_workspace_bytes(rows, width), dtype=torch.uint8, device="cuda")

    def forward(self, tokens):
        self.x = self.embedding[tokens]
        mp.mp_layernorm_forward(self.y, self.x, self.weight, self.bias, EPS, mean=self.mean, rstd=self.rstd)
        return self.y @ self.output.t()

    def backward_and_step(self, tokens, d_logits):
        torch.matmul(d_logits.t(), self.y, out=self.d_output)
        d_y = d_logits @ self.output
        mp.mp_layernorm_backward(self.d_x, self.d_weight, self.d_bias, d_y, self.x, self.weight, self.mean, self.rstd,
                                 workspace=self.workspace)
        d_embedding = torch.zeros(self.vocab, self.width, device="cuda").index_add_(0, tokens, self.d_x.float())
        self.d_embedding.copy_(d_embedding)
        self.t += 1
        self.opt.step(self.params, self.grads, self.master, self.m, self.v, t=self.t, seed=self.t)


def train(steps=300, seed=0, rows=1024, vocab=1003, top=16):
    """Mean losses over the first and the last hundredth of the steps, of the teacher and of the student."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    follow = torch.randint(0, vocab, (vocab, 4), generator=gen, device="cuda")  # a token's four likely successors

    def batch():
        tokens = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
        pick = torch.randint(0, 4, (rows,), generator=gen, device="cuda")
        return tokens, follow[tokens, pick]

    f = dict(device="cuda")
    logp, lse, entropy = torch.empty(rows, **f), torch.empty(rows, **f), torch.empty(rows, **f)
    top_logp, top_index = torch.empty(rows, top, **f), torch.empty(rows, top, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    teacher = Head(vocab, 256, rows, 3e-3, seed)
    d_logp = torch.full((rows,), -1.0 / rows, **f)  # loss = mean of -log p
    teacher_loss = []
    for _ in range(steps):
        tokens, target = batch()
        logits = teacher.forward(tokens)
        mp.mp_token_logprob_forward(logits, target, logp=logp, lse=lse, entropy=entropy, d_status=status)
        teacher_loss.append(-logp.mean())
        mp.mp_token_logprob_backward(logits, logits, target, lse=lse, dlogp=d_logp)  # over the logits
        teacher.backward_and_step(tokens, logits)

    student = Head(vocab, 128, rows, 3e-3, seed + 1)
    loss, weight = torch.empty(rows, **f), torch.full((rows,), 1.0 / rows, **f)
    student_loss = []
    for _ in range(steps):
        tokens, _ = batch()
        mp.mp_token_logprob_forward(teacher.forward(tokens), top_logp=top_logp, top_index=top_index)
        logits = student.forward(tokens)
        mp.mp_distill_topk(loss, logits, logits, top_logp.to(logits.dtype), top_index, row_weight=weight,
                           d_status=status)  # over the logits
        student_loss.append(loss.sum())
        student.backward_and_step(tokens, logits)
    teacher.opt.check_status()
    student.opt.check_status()
    if int(status):
        raise mp.MpError(int(status), "train_head")
    k = max(1, steps // 100)

    def ends(x):
        x = torch.stack(x)
        return float(x[:k].mean()), float(x[-k:].mean())
    return ends(teacher_loss), ends(student_loss)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    teacher, student = train(a.steps, a.seed)
    print("teacher, cross entropy:    %.3f -> %.3f" % teacher)
    print("student, divergence of it: %.3f -> %.3f" % student)


if __name__ == "__main__":
    main()
