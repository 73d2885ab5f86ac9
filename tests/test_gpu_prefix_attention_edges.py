"""Attention over a shared prefix where a row, a cached token or a length is
not as it should be, on the GPU against the 64-bit form."""
import math

import pytest
import torch

from fp8_w8a8_dynamic_b200 import mfp8
from serving_ref import Batch

pytestmark = pytest.mark.gpu

PATHS = (mfp8.ATTEND_ROWS, mfp8.ATTEND_TALL)
ALL_PATHS = (mfp8.ATTEND_AUTO,) + PATHS


@pytest.fixture(autouse=True)
def status_stays_clean():
    yield
    assert mfp8.device_status() == mfp8.OK


def run(b, path, **kw):
    out, lse = mfp8.prefix_attention(*b.args(), want_lse=True, path=path, **kw)
    return out, lse, b.D ** -0.5


# ------------------------------------------- a query row that is not finite --

@pytest.mark.parametrize("path", ALL_PATHS)
@pytest.mark.parametrize("D", (64, 128))
def test_one_infinite_element_makes_its_row_nan(D, path):
    """Every product with an infinity is infinite or NaN, so the softmax has no
    value, however small the keys; the other rows keep their bits."""
    b = Batch([1] * 80, [9, 700] * 40, 6000, 8, 2, D, 64, seed=31, k_gain=2.0 ** -6)
    want, want_lse, _ = run(b, path)
    bad = [(17, 3, 5, math.inf), (40, 0, D - 1, -math.inf), (41, 7, 0, math.nan), (79, 2, D // 2, math.inf)]
    keep = torch.ones(80, 8, dtype=torch.bool, device="cuda")
    for t, h, d, x in bad:
        b.q[t, h, d] = x
        keep[t, h] = False
    got, lse, _ = run(b, path)
    assert got[~keep].isnan().all() and lse[~keep].isnan().all()
    assert torch.equal(got[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])


@pytest.mark.parametrize("path", PATHS)
def test_an_infinite_row_whose_only_logit_is_minus_infinity(path):
    """It sees a token, so it is not a row that sees nothing."""
    b = Batch([1, 1], [1, 1], 0, 1, 1, 128, 8, seed=32)
    key = b.values(b.slots[1], 0)[0][0]
    d = int(key.abs().argmax())
    b.q[0, 0, d] = -math.inf if key[d] > 0 else math.inf
    out, lse, _ = run(b, path)
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert out[1].isfinite().all() and lse[1].isfinite().all()


@pytest.mark.parametrize("path", PATHS)
def test_an_infinite_row_that_sees_nothing(path):
    b = Batch([1, 3], [0, 2], 0, 8, 2, 128, 16, seed=33)
    b.q[0, 1, 3] = math.inf
    b.q[1, 5, 9] = math.nan  # the first of three new tokens with two cached: before both
    out, lse, scale = run(b, path)
    b.check(out, lse, scale)
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all()
