"""Pins for the oracle's linear layers and layer norms, a ciphertext a feature,
and the binding's host checks of the same calls (no GPU work).

Checked on encrypted slots against float64:
  * the product with an 8-bit matrix with scales for each channel (either side)
    and each token, and bias; and, word for word, against Python integers;
  * sums and variance, the normalised input, gamma and beta, with the
    polynomial for 1 / sqrt in between;
  * the gradients, against the formula's and against central differences.

Tolerance: 2^-20 of the largest value, the project's bound for decrypted
results.  Every encryption, key switch and rescale adds an error of about
sqrt(N h) sigma < 2^11 in units of one coefficient (N = 2^10, h = 64, sigma =
3.2) and a decode sums N coefficients in quadrature (2^5): 2^(11 + 5 - 50) =
2^-34 of a unit value at the scale of 2^50.  The product multiplies it by sum
|w| scale < 16 * 2^7 * 2^-5 = 2^6; sums over F = 6 features and the factor F
of the sums by F^2 < 2^6; the polynomial's slope is below 1; the gradient's
products meet factors of at most 2^3 (F |g|, xhat): below 2^-34 2^12 = 2^-22 of
a unit value, and every output's largest value is at least 1/2."""
import numpy as np
import pytest

import ckks_synth as S
from helpers import encrypt_slots, galois_key, params, rel_err, relin_key, secret
from linear_util import differences, features, norm_backward, norm_forward, rsqrt_poly

TOL = 2.0 ** -20


class Scheme:
    """Keys and encryption for one small parameter set (50-bit primes near the scale)."""

    def __init__(self, orc, L, dnum):
        self.orc, self.P = orc, params(orc, 10, L, 50, -(-L // dnum), 60, dnum)
        self.n = self.P.N // 2
        self.s, self.s_ntt = secret(orc, self.P, 9, 64)
        self.rlk = relin_key(orc, self.P, self.s_ntt, 9)
        self.scale = 2.0 ** 50

    def enc(self, z, level, tag, scale=None):
        return encrypt_slots(self.orc, self.P, self.s_ntt, np.asarray(z, dtype=np.complex128), scale or self.scale,
                             level, 9, tag)

    def dec(self, ct, scale):
        return self.orc.decrypt(self.P, ct.shape[-2] - 1, ct, self.s_ntt, scale).real

    def steps(self, radices):
        gal, keys, stride = [], [], 1
        for r in radices:
            g = [self.P.galois(stride * k) for k in range(1, r)]
            gal.append(g)
            keys.append([galois_key(self.orc, self.P, self.s_ntt, v, 9, "g%d" % v) for v in g])
            stride *= r
        return gal, keys


@pytest.fixture(scope="module")
def sch(orc):
    return Scheme(orc, 13, 3)


@pytest.mark.parametrize("B,n_in,n_out", [(1, 1, 1), (2, 5, 3)])
def test_matmul_words(orc, sch, B, n_in, n_out):
    """Sums of integer multiples modulo every prime, from Python integers."""
    P = sch.P
    x = S.uniform_limbs(S.stream(1, "mm"), P.q[:2], P.N, lead=(B, n_in, 2))
    w = S.stream(1, "w").integers(-128, 128, (n_out, n_in)).astype(np.int8)
    got, scale = orc.matmul_i8(P, 1, x, w, 3.0)
    assert scale == 3.0
    big = x.astype(object)
    for b in range(B):
        for j in range(n_out):
            acc = sum(int(w[j, i]) * big[b, i] for i in range(n_in))
            for limb in range(2):
                assert np.array_equal(got[b, j, :, limb], (acc[:, limb] % P.q[limb]).astype(np.uint64))


@pytest.mark.parametrize("scale_in", [False, True])
@pytest.mark.parametrize("token", [False, True])
def test_matmul_decrypts_to_the_layer(orc, sch, scale_in, token):
    n, n_in, n_out, lv = sch.n, 16, 3, 4
    rng = S.stream(2, "layer")
    x, w = rng.uniform(-1, 1, (n_in, n)), rng.integers(-127, 128, (n_out, n_in)).astype(np.int8)
    sc, bias = rng.uniform(0.01, 0.03, n_in if scale_in else n_out), rng.normal(0, 1, n_out)
    tok = rng.uniform(0.5, 1, n) * (np.arange(n) % 7 != 0)  # every seventh token is padding
    ct = np.stack([sch.enc(v, lv, "x%d" % i) for i, v in enumerate(x)])[None]
    pt = orc.encode(sch.P, tok.astype(np.complex128), sch.scale, lv)[None] if token else None
    y, s = orc.matmul_i8(sch.P, lv, ct, w, sch.scale, sc, scale_in, pt, sch.scale, bias)
    ref = w.astype(float) @ (sc[:, None] * x) if scale_in else sc[:, None] * (w.astype(float) @ x)
    ref = ref * (tok if token else 1) + bias[:, None]
    for j in range(n_out):
        assert rel_err(sch.dec(y[0, j], s), ref[j]) < TOL


def test_layer_norm_and_gradients(orc, sch):
    P, n, F, eps, pad = sch.P, sch.n, 6, 1e-3, 9
    rng = S.stream(3, "norm")
    coeffs, fit = rsqrt_poly(0.4)
    x = features(rng, F, n, pad, 0.4, eps)
    gamma, beta = rng.uniform(0.5, 1.5, F), rng.normal(0, 1, F)
    lv = 12
    ct = np.stack([sch.enc(v, lv, "nx%d" % i) for i, v in enumerate(x)])[None]
    # eps - 1: the polynomial takes u = variance + eps - 1
    s, u = orc.layernorm_var(P, lv, ct, sch.scale, eps - 1, sch.rlk)
    assert rel_err(sch.dec(s[0], sch.scale), x.sum(0)) < TOL
    ref_u = x.var(0) + eps - 1
    assert rel_err(sch.dec(u[0], sch.scale), ref_u) < TOL
    r, s_r = orc.poly_eval_tree(P, lv - 2, u, sch.scale, coeffs, sch.rlk)
    ref_r = np.polynomial.polynomial.polyval(ref_u, coeffs)
    assert rel_err(sch.dec(r[0], s_r), ref_r) < TOL
    y = orc.layernorm(P, ct, s, r, sch.scale, s_r, gamma, beta, sch.rlk)
    xh = orc.layernorm(P, ct, s, r, sch.scale, s_r, None, None, sch.rlk)
    ref_xh = norm_forward(x, ref_r)
    for i in range(F):
        assert rel_err(sch.dec(xh[0, i], sch.scale), ref_xh[i]) < TOL
        assert rel_err(sch.dec(y[0, i], sch.scale), gamma[i] * ref_xh[i] + beta[i]) < TOL
    # backward: gradients of zero keep the padded tokens out
    lg = xh.shape[-2] - 1
    assert lg == 5
    dy = rng.uniform(-1, 1, (F, n)) * (np.arange(n) < n - pad)
    dct = np.stack([sch.enc(v, lg, "dy%d" % i) for i, v in enumerate(dy)])[None]
    gal, keys = sch.steps([4, 8, 16])
    out = orc.layernorm_grad(P, lg, dct, xh, r, sch.scale, s_r, gamma, sch.rlk, gal, keys)
    ref_dx, size = norm_backward(dy, ref_xh, ref_r, gamma)
    dif = differences(x[:, : n - pad], dy[:, : n - pad], gamma, beta, eps)
    for i in range(F):
        dx = sch.dec(out["dx"][0, i], sch.scale)
        assert rel_err(dx, ref_dx[i]) < TOL
        # differences of the layer norm itself, whose 1 / sqrt the polynomial meets to `fit`: rstd enters dx up to
        # three times (itself, and xhat twice); the differences' own error is h^2 and 2^-53 / h in units of the loss
        assert np.max(np.abs(dx[: n - pad] - dif[i])) < 4 * fit * size + 1e-8 + TOL * size
        # the sum over 512 slots, in every slot; its terms' errors add to at most 512 times a term's, and its largest
        # value is compared with the terms' sum of sizes
        dg = sch.dec(out["dgamma"][i], sch.scale ** 2 / float(P.q[lg]))
        terms = dy[i] * ref_xh[i]
        assert np.max(np.abs(dg - terms.sum())) < TOL * np.abs(terms).sum()
        db = sch.dec(out["dbeta"][i], sch.scale)
        assert np.max(np.abs(db - dy[i].sum())) < TOL * np.abs(dy[i]).sum()


@pytest.fixture(scope="module")
def lib():
    import private_rns_ckks_amd as L

    return L


def test_binding_checks_arguments(lib):
    """Raised on the host before the library is called."""
    torch = pytest.importorskip("torch")

    class Ctx:  # what the checks read of a context
        N, L, device, key_words, handle = 1024, 4, 0, 3 * 2 * 6 * 1024, None

    cpu = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(lib.ArgumentError):
        lib.ckks_matmul_i8(Ctx, cpu, 1, 1, cpu, 1, 1, 1.0, cpu)
    with pytest.raises(lib.ArgumentError):
        lib.ckks_layernorm_var(Ctx, cpu, 1, 1, 2, 1.0, 0.0, cpu, cpu, cpu)
    with pytest.raises(lib.ArgumentError):
        lib.ckks_layernorm(Ctx, cpu, cpu, 1, 1, 2, 1.0, cpu, 2, 1.0, None, None, cpu, cpu)
    with pytest.raises(lib.ArgumentError):
        lib.ckks_layernorm_grad(Ctx, cpu, 1, 1, 2, cpu, 2, 1.0, cpu, 2, 1.0, None, cpu, None, d_dx=cpu)
    with pytest.raises(lib.ArgumentError):
        lib._doubles([1.0, 2.0], 3, "scales")
    assert list(lib._doubles(np.array([1.5, -2.0]), 2, "scales")) == [1.5, -2.0]
    assert list(lib._doubles([1, 2.5], 2, "scales")) == [1.0, 2.5]
    assert list(lib._doubles(np.array([1, 2], dtype=np.float32), 2, "scales")) == [1.0, 2.0]
    assert list(lib._doubles(np.arange(6.0)[::2], 3, "scales")) == [0.0, 2.0, 4.0]
    assert lib._doubles(None, 3, "scales") is None


def test_flags_match_the_header(lib):
    import os
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ckks.h")).read()
    for name in ("CKKS_W_TRANSPOSED", "CKKS_SCALE_IN"):
        assert int(re.search(r"#define %s (\d+)u" % name, text).group(1)) == getattr(lib, name)
