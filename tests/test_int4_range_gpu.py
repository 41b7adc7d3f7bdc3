"""The INT4 cache at the ends of its numbers: V rows whose scales lie far apart, channels of zeros, NaN rows, queries of
any magnitude, and the quantiser's scale where the range of a row is no fp32 number."""
import numpy as np
import pytest

from tests import _int4 as I4
from tests.test_int4_gpu import _check_decode, _decode

pytestmark = pytest.mark.gpu


def _set_row(cache, which, b, h, pos, word, codes=None):
    """Word (and packed codes) of one row of request b."""
    pid, slot = cache.table[b, pos // cache.P], pos % cache.P
    cache.words[which, pid, h, slot] = word
    if codes is not None:
        cache.pools[which][pid, h, slot] = codes


# ---------------------------------------------------------------------------- weights and zero points
@pytest.mark.parametrize("d", [64, 128])
def test_a_channel_of_zeros_comes_out_near_zero(d):
    """V elements with c = z = 15 under weights that f16 rounds by 2^-13 of their value, all to the same side: a product
    with rounded weights less zero points under others would leave 15 times that. What may be left: the 16 products of an
    MMA and its accumulator are added with an error of 17 units of 2^-23 of the sum, 16 MMAs in a row; the zero points'
    share, added in fp32, 2^-19; both of sums that come to 15 times the weights."""
    L = 256
    cache = I4.Cache([L], Hkv=1, d=d, P=16, seed=109)
    cache.words[0] = 0x3F88
    cache.pools[0][:] = 0x88                                 # K is zero
    _set_row(cache, 0, 0, 0, 3, 0x3F88, np.array([0x89] + [0x88] * (d // 2 - 1)))   # but for one element
    cache.words[1] = 0x3F8F                                  # V: scale 1, zero point 15
    cache.pools[1][..., ::2] |= 0x0F                         # channels 0, 4, 8 ..: zero
    p = np.exp(-0.3)
    assert abs(float(np.float16(p)) / p - 1) > 2.0 ** -13
    q = np.zeros((1, 1, 1, d))
    q[..., 0] = 1.0
    out, lse = _decode(cache, q, 1, tile=256, sm_scale=0.3)
    _check_decode(cache, q, 1, out, lse, sm_scale=0.3)
    assert np.abs(out[..., ::4]).max() <= 15 * (17 * 16 * 2.0 ** -23 + 2.0 ** -19)
