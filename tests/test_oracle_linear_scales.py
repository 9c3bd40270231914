"""How far the rounded constants of the layer norm calls move their results'
scales, on the oracle (no GPU work).

The ciphertexts are trivial (c1 = 0), so no encryption and no key switch adds
an error and what is left is rounding: an encoded coefficient and a rescaled
one are each off by at most 1/2, evenly spread, so a slot is off by sqrt(N /
12) = 9.3 in the square mean and, over 512 slots, by less than 5 times that,
2^5.6.  At the scale of 2^30 that is 2^-24.4."""
import numpy as np
import pytest

import ckks_synth as S
from helpers import params
from linear_util import features

SCALE, LEAST = 2.0 ** 30, 2 ** 19  # of unit values; the least constant that the library takes


@pytest.fixture(scope="module")
def P(orc):
    return params(orc, 10, 5, 30, 1, 60, 5)


def variance_error(orc, P, F):
    """(constant k, largest error of the variance relative to the largest variance)."""
    n, lv = P.N // 2, 4  # the variance keeps three limbs: one does not hold 2^30 of a unit value
    x = features(S.stream(1, "scales"), F, n, 0, 0.4, 0.0)
    ct = np.stack([np.stack([pt, np.zeros_like(pt)]) for pt in
                   (orc.encode(P, v.astype(np.complex128), SCALE, lv) for v in x)])[None]
    rlk = S.uniform_limbs(S.stream(1, "scales/key"), P.mods, P.N, lead=(P.dnum, 2))
    _, var = orc.layernorm_var(P, lv, ct, SCALE, 0.0, rlk)
    got = orc.decrypt(P, lv - 2, var[0], orc.secret_ntt(P, np.zeros(P.N, dtype=np.int64)), SCALE).real
    k = orc.whole(float(P.q[4]) * float(P.q[3]) / (float(F) * float(F)) / SCALE)
    return k, float(np.max(np.abs(got - x.var(0))) / np.max(x.var(0)))


@pytest.mark.parametrize("F", [6, 32, 45])
def test_variance_keeps_its_scale_from_the_least_constant_on(orc, P, F):
    """k >= 2^19: its rounding is 2^-20 at most; the inputs' rounding enters by 2 mean |x - mean| < 2, the
    rescales' (the second's, and the first's over a prime) once: 3 * 2^-24.4 of variances of 0.6 to 1.4."""
    k, err = variance_error(orc, P, F)
    assert k >= LEAST
    assert err < 0.5 / k + 3 * 2.0 ** -24.4


def test_variance_loses_its_scale_below(orc, P):
    """768 features on 30-bit primes: k = 1820 for 1820.2, and the rounding is all of the error."""
    k, err = variance_error(orc, P, 768)
    assert k < LEAST
    q = float(P.q[4]) * float(P.q[3]) / (768.0 * 768.0) / SCALE
    off = abs(k / q - 1)
    assert off > 2.0 ** -14
    assert abs(err - off) < 3 * 2.0 ** -24.4
