"""Limits of the training-head operators' arguments (no GPU needed: every call
here is refused, or has nothing to do, before any device work)."""
import pytest

from test_train_args import DST, LNB, LPB, LPF, call, mp  # noqa: F401


@pytest.mark.parametrize("name,base", [("mp_token_logprob_forward", LPF), ("mp_token_logprob_backward", LPB),
                                       ("mp_distill_topk", DST)])
def test_scale_limit(mp, name, base):  # noqa: F811
    # scale * log2(e) has to be finite in fp32
    for scale, status in ((2.0 ** 126, mp.MP_OK), (2.0 ** 126 * (1 + 2.0 ** -23), mp.MP_ERR_RANGE),
                          (3e38, mp.MP_ERR_RANGE), (2.0 ** -149, mp.MP_OK)):
        assert call(mp, name, list(base), base, rows=0, scale=scale) == status, scale


def test_layernorm_backward_of_no_rows(mp):  # noqa: F811
    # tensors without elements have no address; dx of no rows is nothing to do
    none = dict(rows=0, dx=None, dy=None, x=None, mean=None, rstd=None)
    assert call(mp, "mp_layernorm_backward", list(LNB), LNB, dweight=None, dbias=None, **none) == mp.MP_OK
    assert call(mp, "mp_layernorm_backward", list(LNB), LNB, dweight=None, dbias=None, **{**none, "rows": 1}) == mp.MP_ERR_NULL
    assert call(mp, "mp_layernorm_backward", list(LNB), LNB, dweight=None, dbias=None, **{**none, "d": 0}) == mp.MP_ERR_RANGE
