"""The block's operators together, as the example runs them: its gradients, with
everything in fp32 but what is kept in 8 bits, against 64-bit autograd of the
same function from the same kept values."""
import importlib.util
import math
import os

import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod



def reference(model, tokens, target):
    """Loss and gradients in 64 bits, autograd throughout. The values kept in 8 bits enter the backward pass as
    constants: each operator is written as its own Function with the formula of its gradient."""
    def norm(h, kept, w):
        class Norm(torch.autograd.Function):
            @staticmethod
            def forward(ctx, h, w):
                r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + model_eps)
                ctx.save_for_backward(r, w)
                return h * r * w

            @staticmethod
            def backward(ctx, dy):
                r, w = ctx.saved_tensors
                xh, g = kept * r, dy * w
                return r * (g - xh * (g * xh).mean(1, keepdim=True)), (dy * xh).sum(0)
        return Norm.apply(h, w)

    def gated(a, b, ka, kb):
        class Gated(torch.autograd.Function):
            @staticmethod
            def forward(ctx, a, b):
                return a * torch.sigmoid(a) * b

            @staticmethod
            def backward(ctx, dy):
                s = torch.sigmoid(ka)
                return dy * kb * (s + ka * s * (1 - s)), dy * ka * s
        return Gated.apply(a, b)

    model_eps = 1e-5
    p = {k: v.double().requires_grad_() for k, v in model.p.items()}
    H, K, D, B, T = model.heads, model.kv_heads, model.dim, model.batch, model.length
    kept = [R.unpack(*s) for s in model.h8]
    x = p["embedding"][tokens.view(-1)]
    qkv = (norm(x, kept[0], p["norm1"]) @ p["wqkv"].t()).view(B, T, H + 2 * K, D)
    f = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    angle = torch.arange(T, dtype=torch.float64, device="cuda")[:, None] * f
    c, s = torch.cos(angle)[None, :, None], torch.sin(angle)[None, :, None]

    def turn(v):
        a, b = v[..., :D // 2], v[..., D // 2:]
        return torch.cat((a * c - b * s, a * s + b * c), -1)

    q, k, v = turn(qkv[:, :, :H]), turn(qkv[:, :, H:H + K]), qkv[:, :, H + K:]
    k, v = (t.repeat_interleave(H // K, 2) for t in (k, v))
    scores = torch.einsum("bthd,bshd->bhts", q, k) * D ** -0.5
    prob = torch.softmax(scores.masked_fill(~model.mask, -math.inf), 3)
    mixed = torch.einsum("bhts,bshd->bthd", prob, v).reshape(B * T, H * D)
    h = x + mixed @ p["wo"].t()
    both = norm(h, kept[1], p["norm2"]) @ p["gate_up"].t()
    n = model.inner
    # the product behind the activation has its weight gradient from the output computed again from the 8 bits
    ka, kb = R.unpack(*model.gate8), R.unpack(*model.up8)
    again = ka * torch.sigmoid(ka) * kb

    class Down(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, w):
            ctx.save_for_backward(w)
            return a @ w.t()

        @staticmethod
        def backward(ctx, dy):
            return dy @ ctx.saved_tensors[0], dy.t() @ again

    h = h + Down.apply(gated(both[:, :n], both[:, n:], ka, kb), p["down"])
    logits = norm(h, kept[2], p["norm3"]) @ p["output"].t()
    loss = -torch.log_softmax(logits, 1).gather(1, target[:, None]).mean()
    loss.backward()
    return float(loss.detach()), {k: v.grad for k, v in p.items()}


def test_gradients(example):
    import mixed_precision_adamw_gb300 as mp
    torch.backends.cuda.matmul.allow_tf32 = False
    model = example.Block(vocab=211, width=96, heads=6, kv_heads=2, inner=161, batch=2, length=37, seed=3,
                          dtype=torch.float32)
    with torch.no_grad():
        for name in model.p:
            model.p[name].mul_(8.0 if model.p[name].dim() == 2 else 1.0)  # activations of ordinary size
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randint(0, 211, (2, 37), generator=g, device="cuda")
    target = torch.randint(0, 211, (74,), generator=g, device="cuda")
    logits = model.forward(tokens)
    logp, lse = torch.empty(74, device="cuda"), torch.empty(74, device="cuda")
    mp.mp_token_logprob_forward(logits, target, logp=logp, lse=lse)
    mp.mp_token_logprob_backward(logits, logits, target, lse=lse, dlogp=torch.full((74,), -1.0 / 74, device="cuda"))
    model.backward(tokens, logits)
    torch.cuda.synchronize()
    loss, ref = reference(model, tokens, target)
    assert abs(-float(logp.mean()) - loss) <= 1e-5 * loss
    for name, want in ref.items():
        got = model.g[name].double()
        # some forty fp32 roundings on the way, each entering through sums of at most a few hundred terms of both
        # signs: 40 sqrt(300) u is 4e-5 of a tensor's norm
        assert float((got - want).norm()) <= 4e-5 * float(want.norm()), name


def test_example_runs(example):
    first, last = example.train(steps=3)
    assert math.isfinite(first) and math.isfinite(last)
