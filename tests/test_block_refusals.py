"""Calls of a block's operators that are refused although each argument alone is
right: a buffer that is given for two things; and a size beyond 32 bits (no GPU
needed: refused before any device work)."""
import pytest

from test_block_args import GF, RF, RO
from test_train_args import FAKE, call, mp  # noqa: F401


@pytest.mark.parametrize("kw", [dict(q_out=4 * FAKE), dict(k_out=2 * FAKE), dict(q_out=4 * FAKE, k_out=2 * FAKE)])
def test_rope_over_the_other_input(mp, kw):  # noqa: F811
    # whose heads other blocks have yet to read
    assert call(mp, "mp_rope", list(RO), RO, **kw) == mp.MP_ERR_RANGE
    no_keys = {**RO, "k_heads": 0, "k_out": None}  # then nobody reads them
    assert call(mp, "mp_rope", list(RO), no_keys, q_out=4 * FAKE, turns=None) == mp.MP_ERR_NULL


@pytest.mark.parametrize("name,base,kw", [
    ("mp_rmsnorm_forward", RF, dict(y8_scale=2 * FAKE, h8_scale=2 * FAKE)),
    ("mp_rmsnorm_forward", RF, dict(y8_scale=2 * FAKE, h8_scale=2 * FAKE, y8_kind=2)),
    ("mp_gated_forward", GF, dict(gate8_scale=6 * FAKE, up8_scale=6 * FAKE)),
])
def test_one_buffer_for_both_scales(mp, name, base, kw):  # noqa: F811
    assert call(mp, name, list(base), base, **kw) == mp.MP_ERR_RANGE


@pytest.mark.parametrize("rotary_dim", [(1 << 32) + 64, 1 << 40, 1 << 70, -(1 << 32) + 64])
def test_rotary_dim_beyond_32_bits(mp, rotary_dim):  # noqa: F811
    with pytest.raises(mp.MpError) as e:
        mp.mp_rope_frequencies(rotary_dim, device="cpu")
    assert e.value.status == mp.MP_ERR_RANGE
