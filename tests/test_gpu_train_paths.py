"""The training-head operators on the paths that sizes, masks and alignment
select, beyond tests/test_gpu_train_ops.py: against the same 64-bit references
and bounds (tests/train_ref.py)."""
import math

import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu

BF, HF, FF = torch.bfloat16, torch.float16, torch.float32
INF = math.inf


@pytest.fixture(scope="module")
def mp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    import mixed_precision_adamw_gb300 as mp
    return mp


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, g, std=1.0, dtype=FF):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def f32(*shape, fill=-7.0):
    return torch.full(shape, fill, dtype=FF, device="cuda")


# --- rows split over the blocks of a cluster --------------------------------------

@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("rows,vocab", [(1, 4100), (1, 8200), (3, 16391), (1, 128256), (37, 50304), (75, 20001)])
def test_logprob_clusters_started_one_after_the_other(mp, rows, vocab, dtype):
    # calls in flight on two streams, each cluster's blocks taking what the other leaves free:
    # the blocks of a row start and finish at different times
    g = gen(rows + vocab)
    x = randn((rows, vocab), g, 2.5, dtype)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for i in range(60):
        o = (f32(rows), f32(rows), f32(rows), f32(rows, 8),
             torch.full((rows, 8), -9, dtype=torch.int32, device="cuda"))
        torch.cuda.current_stream().synchronize()  # the fills, before another stream writes
        mp.mp_token_logprob_forward(x, t, logp=o[0], lse=o[1], entropy=o[2], top_logp=o[3], top_index=o[4],
                                    stream=streams[i % 2])
        outs.append(o)
    torch.cuda.synchronize()
    ref, tol = R.lp_forward(x, t, 1.0, 8)
    for name, got in zip(("logp", "lse", "entropy", "top_logp"), outs[0]):
        R.assert_within(got, ref[name], tol[name], f"{rows}x{vocab} {dtype} {name}")
    assert torch.equal(outs[0][4], ref["top_index"])
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))
