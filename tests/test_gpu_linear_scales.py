"""Scales that the linear layer and layer norm calls refuse, and the nearest
that they take: those give the oracle's words."""
import numpy as np
import pytest

import ckks_synth as S
from gpu_util import announce, empty_dev, make_pair, to_dev, torch_cuda
from test_gpu_linear import int8_dev, key, same, words

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** 19  # of a constant that sets a result's scale


@pytest.fixture(scope="module")
def lib():
    torch_cuda()
    import private_rns_ckks_amd as L

    return L


@pytest.fixture(scope="module")
def pair(lib, orc):
    """30-bit primes: products of two scales leave little room for the number of features."""
    ctx, P = make_pair(lib, orc, 10, 7, 30, 3, 60, 3)
    yield ctx, P
    ctx.close()


def refused(lib, fn, *a, **kw):
    with pytest.raises(lib.CKKSError) as e:
        fn(*a, **kw)
    assert e.value.code == lib.CKKS_EINVAL, str(e.value)


@pytest.mark.parametrize("F,lv", [(1, 6), (5, 2)])
def test_variance_constant(lib, orc, pair, F, lv):
    ctx, P = pair
    announce("least constant of the variance, F=%d" % F)
    x, rlk = words(P, 1, "x", lv + 1, (1, F, 2)), key(P, 1, "rlk")
    d_x, d_k, d_s, d_v = to_dev(x), to_dev(rlk), empty_dev((1, 2, lv + 1, P.N)), empty_dev((1, 2, lv - 1, P.N))
    d_v.fill_(-7)
    room = float(P.q[lv]) * float(P.q[lv - 1]) / F ** 2
    refused(lib, lib.ckks_layernorm_var, ctx, d_x, 1, F, lv, room / (LEAST - 1), 0.5, d_k, d_s, d_v)
    assert bool((d_v == -7).all())
    lib.ckks_layernorm_var(ctx, d_x, 1, F, lv, room / LEAST, 0.5, d_k, d_s, d_v)
    s, v = orc.layernorm_var(P, lv, x, room / LEAST, 0.5, rlk)
    same(d_s, s, "sum")
    same(d_v, v, "var")


def test_variance_of_many_features_on_small_primes(lib, pair):
    """The scale of 2^30 on 30-bit primes: 45 features have room, 46 and 768 not."""
    ctx, P = pair
    announce("features on small primes")
    lv = 2
    d_x, d_k = empty_dev((1, 768, 2, lv + 1, P.N)).zero_(), to_dev(key(P, 2, "rlk"))
    d_s, d_v = empty_dev((1, 2, lv + 1, P.N)), empty_dev((1, 2, lv - 1, P.N))
    lib.ckks_layernorm_var(ctx, d_x, 1, 45, lv, 2.0 ** 30, 0.0, d_k, d_s, d_v)
    for F in (46, 768):
        refused(lib, lib.ckks_layernorm_var, ctx, d_x, 1, F, lv, 2.0 ** 30, 0.0, d_k, d_s, d_v)


@pytest.mark.parametrize("affine", [False, True])
def test_norm_constant(lib, orc, pair, affine):
    """Before gamma: a weight may be as small as the caller likes."""
    ctx, P = pair
    announce("least constant of the norm, affine=%s" % affine)
    F, lv, t = 3, 5, 3
    x, rlk, r, s = words(P, 3, "x", lv + 1, (1, F, 2)), key(P, 3, "rlk"), words(P, 3, "r", t + 1, (1, 2)), words(
        P, 3, "s", lv + 1, (1, 2))
    gamma, beta = (np.array([1e-9, 1.0, -0.5]), np.ones(F)) if affine else (None, None)
    d = [to_dev(v) for v in (x, s, r, rlk)]
    y = empty_dev((1, F, 2, t - 1, P.N))
    room = float(P.q[t]) * float(P.q[t - 1]) / F
    refused(lib, lib.ckks_layernorm, ctx, d[0], d[1], 1, F, lv, 2.0 ** 30, d[2], t, room / (LEAST - 1), gamma, beta, d[3], y)
    lib.ckks_layernorm(ctx, d[0], d[1], 1, F, lv, 2.0 ** 30, d[2], t, room / LEAST, gamma, beta, d[3], y)
    same(y, orc.layernorm(P, x, s, r, 2.0 ** 30, room / LEAST, gamma, beta, rlk))


def test_gradient_constants(lib, orc, pair):
    ctx, P = pair
    announce("least constants of the gradient")
    F, lv = 2, 6
    dy, xh = words(P, 4, "dy", lv + 1, (1, F, 2)), words(P, 4, "xh", lv + 1, (1, F, 2))
    r, rlk = words(P, 4, "r", lv + 1, (1, 2)), key(P, 4, "rlk")
    d = [to_dev(v) for v in (dy, xh, r, rlk)]
    dx, dg = empty_dev((1, F, 2, lv - 4, P.N)), empty_dev((F, 2, lv, P.N))
    q = [float(v) for v in P.q]
    room_k, room_c = q[lv - 3] * q[lv - 4] / F, q[lv] * q[lv - 1] * q[lv - 2]

    def call(fn, least_k, least_c, **out):
        fn(ctx, d[0], 1, F, lv, d[1], lv, (room_c / least_c) ** 0.5, d[2], lv, room_k / least_k, None, d[3], None, **out)

    grad = lib.ckks_layernorm_grad
    call(lambda *a, **kw: refused(lib, grad, *a, **kw), LEAST - 1, LEAST, d_dx=dx)
    call(lambda *a, **kw: refused(lib, grad, *a, **kw), LEAST, LEAST - 1, d_dx=dx)
    call(grad, LEAST, LEAST, d_dx=dx)
    ref = orc.layernorm_grad(P, lv, dy, xh, r, (room_c / LEAST) ** 0.5, room_k / LEAST, None, rlk, [], [], ("dx", "dgamma"))
    same(dx, ref["dx"])
    call(grad, 1, 1, d_dgamma=dg)  # the weights' gradients have no such constant
    same(dg, ref["dgamma"])


@pytest.mark.parametrize("bias", [False, True])
def test_product_scales(lib, orc, pair, bias):
    """A scale that is not positive and finite is refused with or without a bias that it would multiply; a token
    scale only counts with token rows."""
    ctx, P = pair
    announce("scales of a product, bias=%s" % bias)
    n_in, n_out, lv = 3, 2, 2
    x, tok = words(P, 6, "x", lv + 1, (1, n_in, 2)), words(P, 6, "tok", lv + 1, (1,))
    w = np.array([[3, -1, 2], [0, 5, -128]], np.int8)
    d_x, d_t, d_w, y = to_dev(x), to_dev(tok), int8_dev(w), empty_dev((1, n_out, 2, lv + 1, P.N))
    b = np.array([0.5, -2.0]) if bias else None
    y.fill_(-7)

    def call(scale, tok_scale=1.0, d_tok=None, out=y):
        return lib.ckks_matmul_i8(ctx, d_x, 1, n_in, d_w, n_out, lv, scale, out, d_tok=d_tok, n_tok=int(d_tok is not None),
                                  tok_scale=tok_scale, bias=b)

    for bad in (0.0, -1.0, float("nan"), float("inf"), -float("inf")):
        refused(lib, call, bad)
        refused(lib, call, 2.0 ** 30, bad, d_t)
    refused(lib, call, 2.0 ** 600, 2.0 ** 600, d_t)    # an output scale above the largest double
    refused(lib, call, 2.0 ** -600, 2.0 ** -600, d_t)  # and below the smallest
    assert bool((y == -7).all())
    assert call(2.0 ** 30, float("nan")) == 2.0 ** 30
    same(y, orc.matmul_i8(P, lv, x, w, 2.0 ** 30, bias=b)[0])
    low = empty_dev((1, n_out, 2, lv, P.N))
    got = call(2.0 ** 30, 2.0 ** 25, d_t, low)
    ref, s = orc.matmul_i8(P, lv, x, w, 2.0 ** 30, None, False, tok, 2.0 ** 25, b)
    assert got == s
    same(low, ref)


def test_many_features_decrypt_to_the_norm(lib, orc):
    """768 features at 50 bits: the oracle's words, and the normalised input in float64.

    An encryption is off by less than 2^-31 of a unit value in every slot (tests/test_oracle_linear.py: 2^-34 in the
    square mean, times 5 for the largest of them); the variance meets that times 2 mean |x - mean| < 2, the sum 768
    times, and the rescales add as much as an encryption each; the constants are rounded by 2^-31: below 2^-20 of
    the largest values, 1 and more."""
    from helpers import encrypt_slots, relin_key, secret
    from linear_util import features

    announce("768 features, encrypted")
    ctx, P = make_pair(lib, orc, 10, 6, 50, 2, 60, 3)
    F, lv, scale, n = 768, 5, 2.0 ** 50, P.N // 2
    s, s_ntt = secret(orc, P, 5, 64)
    rlk = relin_key(orc, P, s_ntt, 5)
    x = features(S.stream(5, "scales/features"), F, n, 0, 0.4, 1e-3)
    enc = lambda z, l, t: encrypt_slots(orc, P, s_ntt, z.astype(np.complex128), scale, l, 5, t)
    dec = lambda ct: orc.decrypt(P, ct.shape[-2] - 1, ct, s_ntt, scale).real
    ct = np.stack([enc(v, lv, "x%d" % i) for i, v in enumerate(x)])[None]
    r_ref = 1 / np.sqrt(x.var(0) + 1e-3)
    r = enc(r_ref, 3, "r")[None]
    d_x, d_k = to_dev(ct), to_dev(rlk)
    d_s, d_v, d_y = empty_dev((1, 2, lv + 1, P.N)), empty_dev((1, 2, lv - 1, P.N)), empty_dev((1, F, 2, 2, P.N))
    lib.ckks_layernorm_var(ctx, d_x, 1, F, lv, scale, 1e-3, d_k, d_s, d_v)
    lib.ckks_layernorm(ctx, d_x, d_s, 1, F, lv, scale, to_dev(r), 3, scale, None, None, d_k, d_y)
    sm, v = orc.layernorm_var(P, lv, ct, scale, 1e-3, rlk)
    y = orc.layernorm(P, ct, sm, r, scale, scale, None, None, rlk)
    same(d_s, sm, "sum")
    same(d_v, v, "var")
    same(d_y, y, "norm")
    ref_v, ref_y = x.var(0) + 1e-3, (x - x.mean(0)) * r_ref
    assert np.max(np.abs(dec(v[0]) - ref_v)) < 2.0 ** -20 * np.max(ref_v)
    for i in range(0, F, 37):
        assert np.max(np.abs(dec(y[0, i]) - ref_y[i])) < 2.0 ** -20 * np.max(np.abs(ref_y[i]))
    ctx.close()
