"""Copied columns of interleaved rotations, bit by bit."""
import pytest
import torch

from test_gpu_train_ops import BF, FF, HF, gen, mp, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("rot", [2, 4, 6, 8, 14, 18, 26, 30, 32])
def test_rope_interleaved_copies_bits(mp, rot, dtype):  # noqa: F811
    """A head's columns from rotary_dim on keep their bits, whatever they hold, and do not reach the others."""
    turns, _ = mp.mp_rope_frequencies(rot, 10000.0)
    g = gen(rot)
    x = randn((70, 3, 32), g, 1.0, dtype)
    bits = x.view(torch.int32 if dtype == FF else torch.int16)
    special = [0x7F800001, -0x00000001, -0x80000000, 0x7F800000, 0x00000001] if dtype == FF else \
        [0x7F81, 0x7C01, -1, -0x8000, 0x7F80, 0x7C00, 1]
    pick = torch.randint(0, len(special), bits[..., rot:].shape, generator=g, device=x.device)
    bits[..., rot:] = torch.tensor(special, device=x.device, dtype=torch.int64).to(bits.dtype)[pick]
    keep, clean = bits[..., rot:].clone(), x.clone()
    clean[..., rot:] = 0
    o, c = torch.empty_like(x), torch.empty_like(x)
    mp.mp_rope(o, x, None, None, turns, first_position=3, interleaved=True)
    mp.mp_rope(c, clean, None, None, turns, first_position=3, interleaved=True)
    assert torch.equal(o.view(bits.dtype)[..., rot:], keep)
    assert torch.equal(o[..., :rot], c[..., :rot])
    mp.mp_rope(x, x, None, None, turns, first_position=3, interleaved=True)
    assert torch.equal(bits[..., rot:], keep) and torch.equal(x[..., :rot], c[..., :rot])
