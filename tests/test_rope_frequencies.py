"""kv_rope_frequencies at the ends of its arguments' ranges."""
import numpy as np
import pytest

from paged_kv_cache_273_gb300 import pkv

SCALINGS = {"linear": {}, "parts": dict(trained_len=4096, low=1.0, high=32.0), "wavelength": dict(trained_len=8192, low=1.0, high=4.0)}


@pytest.mark.parametrize("scaling", list(SCALINGS))
def test_a_factor_next_to_nothing(scaling):
    """f_i / factor beyond a double's range is no frequency: the call is refused, not answered with
    what a conversion of infinity gives."""
    with pytest.raises(pkv.PkvError) as e:
        pkv.kv_rope_frequencies(64, scaling=scaling, factor=1e-320, **SCALINGS[scaling])
    assert e.value.status == pkv.PKV_ERR_INVALID


@pytest.mark.parametrize("factor", [1e-300, 1e-12, 0.25, 1e12, 1e300])
def test_factors_far_from_one(factor):
    """Words of LINEAR: the fraction of a turn, whole turns left out, to a double's 53 bits."""
    words, m = pkv.kv_rope_frequencies(32, base=10000.0, scaling="linear", factor=factor)
    assert m == 1.0
    for i in range(16):
        turns = 10000.0 ** (-2.0 * i / 32) / factor / (2 * np.pi)
        part = turns - np.floor(turns)                 # a double's own whole turns leave nothing beyond 2^53
        got = int(words[i]) / 2.0 ** 64
        err = abs(got - part)
        assert min(err, 1.0 - err) <= 4 * np.spacing(turns) + 2.0 ** -64
