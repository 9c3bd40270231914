"""Bit-exact parity of the linear layer and layer norm calls (ckks_matmul_i8,
ckks_layernorm_var, ckks_layernorm, ckks_layernorm_grad) against the CPU
oracle, through the C interface: every output word must be equal, so there
are no tolerances.  Words are uniform residues (what encryption makes them), the
top of the residue range, or real encryptions."""
import numpy as np
import pytest

import ckks_synth as S
from gpu_util import announce, empty_dev, make_pair, misaligned_dev, to_dev, to_host, torch_cuda
from helpers import encrypt_slots, galois_key, relin_key, secret

pytestmark = pytest.mark.gpu

# (log_n, L, q_bits, K, p_bits, dnum)
SETS = {
    "tiny": (12, 4, 30, 1, 60, 4),
    "small": (10, 7, 40, 3, 60, 3),
    "q47": (10, 3, 47, 1, 60, 3),
    "q48": (11, 2, 48, 1, 60, 2),
    "q54": (11, 8, 54, 3, 60, 3),
    "q55": (10, 3, 55, 1, 60, 3),
    "q56": (10, 7, 56, 3, 60, 3),
    "q57": (13, 6, 57, 3, 60, 2),
    "mid": (13, 8, 54, 3, 60, 3),
    "wide": (10, 7, 62, 3, 61, 3),
    "wide61": (11, 8, 61, 4, 62, 2),
    "one": (10, 1, 50, 0, 60, 1),
    "deep": (10, 24, 54, 8, 60, 3),
    "full": (16, 8, 54, 3, 60, 3),
}


@pytest.fixture(scope="module")
def lib():
    torch_cuda()
    import private_rns_ckks_amd as L

    return L


@pytest.fixture(scope="module")
def sets(lib, orc):
    made = {}

    def get(name):
        if name not in made:
            made[name] = make_pair(lib, orc, *SETS[name])
        return made[name]

    return get


def words(P, seed, tag, limbs, lead, top=False):
    fn = S.top_limbs if top else S.uniform_limbs
    return fn(S.stream(seed, "linear/" + tag), P.q[:limbs], P.N, lead=lead)


def key(P, seed, tag, top=False):
    fn = S.top_limbs if top else S.uniform_limbs
    return fn(S.stream(seed, "linear/key/" + tag), P.mods, P.N, lead=(P.dnum, 2))


def steps(lib, P, radices, seed=0, stride=1):
    """(library stages, (galois, keys) for the oracle)."""
    gal, host = [], []
    for s, r in enumerate(radices):
        gal.append([P.galois(stride * k) for k in range(1, r)])
        host.append([key(P, seed, "%d.%d" % (s, k)) for k in range(1, r)])
        stride = stride * r % (P.N // 2) or 1
    return lib.RotateSum(gal, [[to_dev(k) for k in ks] for ks in host]), (gal, host)


def same(got, ref, what=""):
    got = to_host(got)
    assert got.shape == ref.shape
    assert np.array_equal(got, ref), "%s: %d words differ" % (what, int((got != ref).sum()))


def int8_dev(w):
    torch = torch_cuda()
    return torch.from_numpy(np.ascontiguousarray(w, dtype=np.int8)).cuda()


def matrix(seed, n_out, n_in, kind="normal"):
    rng = S.stream(seed, "linear/w")
    if kind == "extreme":
        w = rng.choice(np.array([-128, 127], dtype=np.int8), (n_out, n_in))
        w[0] = -128  # the largest sums either way
        w[-1] = 127
        return w
    return np.clip(np.rint(rng.normal(0, 40, (n_out, n_in))), -128, 127).astype(np.int8)


def matmul(lib, orc, ctx, P, level, B, n_in, n_out, scales="out", tok=0, bias=True, transposed=False, top=False,
           kind="normal", seed=0, check=None):
    """One call against the oracle; check: the outputs the oracle computes (all of them by default)."""
    rng = S.stream(seed, "linear/real")
    x = words(P, seed, "x", level + 1, (B, n_in, 2), top)
    w = matrix(seed, n_out, n_in, kind)
    sc = None if scales == "none" else np.exp(rng.normal(-5, 0.5, n_in if scales == "in" else n_out)) * rng.choice(
        [-1, 1], n_in if scales == "in" else n_out)
    tk = words(P, seed, "tok", level + 1, (tok,), top) if tok else None
    bs = rng.normal(0, 1, n_out) if bias else None
    drop = (sc is not None) + (tk is not None)
    out = empty_dev((B, n_out, 2, level + 1 - drop, P.N))
    flags = (lib.CKKS_W_TRANSPOSED if transposed else 0) | (lib.CKKS_SCALE_IN if scales == "in" else 0)
    got = lib.ckks_matmul_i8(ctx, to_dev(x), B, n_in, int8_dev(w.T if transposed else w), n_out, level, 2.0 ** 30, out,
                             scales=sc, d_tok=None if tk is None else to_dev(tk), n_tok=tok, tok_scale=2.0 ** 25, bias=bs,
                             flags=flags)
    rows = list(range(n_out)) if check is None else check
    ref, s = orc.matmul_i8(P, level, x, w[rows], 2.0 ** 30, sc if sc is None or scales == "in" else sc[rows],
                           scales == "in", tk, 2.0 ** 25, None if bs is None else bs[rows])
    assert got == s
    same(out[:, rows].contiguous(), ref, "matmul_i8")


# ---------------------------------------------------------------- matmul_i8

MATMULS = [
    # set, level, blocks, n_in, n_out, scales, token rows, bias, transposed
    ("tiny", 3, 1, 1, 1, "none", 0, False, False), ("tiny", 3, 1, 16, 12, "out", 0, True, False),
    ("tiny", 2, 2, 5, 9, "in", 1, True, True), ("tiny", 0, 1, 3, 2, "none", 0, True, False),
    ("small", 4, 3, 33, 7, "out", 3, True, False), ("small", 1, 1, 64, 31, "in", 0, False, False),
    ("small", 2, 1, 31, 65, "out", 1, False, True), ("small", 6, 1, 2, 3, "none", 1, True, False),
    ("q47", 1, 1, 40, 5, "out", 0, True, False), ("q48", 1, 1, 100, 33, "out", 0, False, True),
    ("q54", 2, 2, 130, 20, "out", 2, True, False), ("q54", 1, 1, 257, 64, "in", 0, True, True),
    ("q54", 7, 1, 8, 17, "none", 0, False, False), ("q55", 1, 1, 70, 40, "out", 0, True, False),
    ("q56", 2, 1, 33, 34, "in", 1, True, False), ("q57", 1, 1, 17, 5, "out", 0, True, False),
    ("mid", 2, 2, 12, 35, "out", 2, True, False), ("wide", 3, 2, 65, 6, "out", 1, True, True),
    ("wide", 1, 1, 128, 32, "in", 0, False, False), ("wide61", 2, 1, 40, 33, "out", 0, True, False),
    ("one", 0, 2, 37, 8, "none", 0, True, False), ("deep", 23, 1, 6, 4, "out", 1, True, False),
    ("q54", 2, 5, 3, 2, "out", 2, True, False),
    # tiles of 64, 128 and 256 outputs, whole and ragged; inputs of one group and a step, and one more
    ("q54", 1, 1, 16, 64, "out", 0, True, False), ("small", 2, 1, 17, 128, "out", 1, True, True),
    ("q54", 1, 1, 128, 129, "out", 0, True, False), ("q54", 1, 2, 129, 256, "in", 0, False, True),
    ("tiny", 1, 1, 300, 257, "in", 0, True, False), ("small", 1, 1, 256, 300, "out", 0, True, False),
    ("q48", 0, 1, 385, 140, "none", 0, True, False), ("wide", 1, 1, 33, 200, "in", 0, True, False),
    ("q56", 1, 1, 31, 150, "out", 0, False, False), ("q47", 2, 1, 20, 190, "out", 1, True, True),
]


@pytest.mark.parametrize("name,level,B,n_in,n_out,scales,tok,bias,transposed", MATMULS)
@pytest.mark.parametrize("top", [False, True])
def test_matmul_parity(lib, orc, sets, name, level, B, n_in, n_out, scales, tok, bias, transposed, top):
    ctx, P = sets(name)
    announce("matmul_i8 %s level=%d B=%d %dx%d %s tok=%d T=%s top=%s" % (name, level, B, n_in, n_out, scales, tok,
                                                                        transposed, top))
    matmul(lib, orc, ctx, P, level, B, n_in, n_out, scales, tok, bias, transposed, top, "extreme" if top else "normal")


# ---------------------------------------------------------------- layer norm

NORMS = [
    # set, level, rstd level, blocks, features
    ("tiny", 3, 2, 1, 12), ("small", 6, 6, 2, 5), ("small", 2, 2, 1, 1), ("q54", 7, 3, 1, 33), ("q57", 5, 4, 2, 3),
    ("mid", 7, 5, 1, 9), ("wide", 6, 5, 2, 7), ("wide61", 7, 2, 1, 10), ("deep", 23, 14, 1, 3), ("q56", 3, 3, 3, 8),
]


@pytest.mark.parametrize("name,level,t,B,F", NORMS)
@pytest.mark.parametrize("top", [False, True])
def test_layernorm_parity(lib, orc, sets, name, level, t, B, F, top):
    ctx, P = sets(name)
    announce("layernorm %s level=%d rstd=%d B=%d F=%d top=%s" % (name, level, t, B, F, top))
    rng, scale = S.stream(3, "linear/norm"), 2.0 ** (SETS[name][2] - 5)
    x, rlk = words(P, 3, "nx", level + 1, (B, F, 2), top), key(P, 3, "rlk", top)
    d_x, d_k = to_dev(x), to_dev(rlk)
    d_sum, d_var = empty_dev((B, 2, level + 1, P.N)), empty_dev((B, 2, level - 1, P.N))
    lib.ckks_layernorm_var(ctx, d_x, B, F, level, scale, 1e-5, d_k, d_sum, d_var)
    s, v = orc.layernorm_var(P, level, x, scale, 1e-5, rlk)
    same(d_sum, s, "sum")
    same(d_var, v, "var")
    r = words(P, 4, "r", t + 1, (B, 2), top)
    for affine in (True, False):
        gamma, beta = (rng.normal(1, 1, F), rng.normal(0, 1, F)) if affine else (None, None)
        out = empty_dev((B, F, 2, t - 1, P.N))
        lib.ckks_layernorm(ctx, d_x, d_sum, B, F, level, scale, to_dev(r), t, scale * 1.25, gamma, beta, d_k, out)
        same(out, orc.layernorm(P, x, s, r, scale, scale * 1.25, gamma, beta, rlk), "affine=%s" % affine)


GRADS = [
    # set, level, xhat level, rstd level, blocks, features, radices, gamma
    ("small", 5, 6, 5, 1, 4, [3], True), ("small", 6, 6, 6, 2, 3, [2, 2], False), ("q54", 5, 5, 7, 3, 9, [4], True),
    ("mid", 7, 7, 7, 1, 3, [], True), ("q57", 5, 5, 5, 2, 2, [2], True), ("wide", 5, 6, 6, 2, 5, [3], True),
    ("wide61", 6, 7, 6, 1, 2, [], False), ("deep", 15, 20, 23, 1, 2, [2], True), ("small", 5, 5, 6, 1, 1, [5], True),
]


@pytest.mark.parametrize("name,level,lx,lr,B,F,radices,affine", GRADS)
@pytest.mark.parametrize("top", [False, True])
def test_layernorm_grad_parity(lib, orc, sets, name, level, lx, lr, B, F, radices, affine, top):
    ctx, P = sets(name)
    announce("layernorm_grad %s level=%d B=%d F=%d %s top=%s" % (name, level, B, F, radices, top))
    st, (gal, keys) = steps(lib, P, radices, seed=5)
    scale = 2.0 ** (SETS[name][2] - 3)
    gamma = S.stream(5, "linear/gamma").normal(1, 1, F) if affine else None
    dy, xh = words(P, 5, "dy", level + 1, (B, F, 2), top), words(P, 5, "xh", lx + 1, (B, F, 2), top)
    r, rlk = words(P, 5, "gr", lr + 1, (B, 2), top), key(P, 5, "rlk", top)
    shape = {"dx": (B, F, 2, level - 4, P.N), "dgamma": (F, 2, level, P.N), "dbeta": (F, 2, level + 1, P.N)}
    out = {k: empty_dev(v) for k, v in shape.items()}
    lib.ckks_layernorm_grad(ctx, to_dev(dy), B, F, level, to_dev(xh), lx, scale, to_dev(r), lr, scale, gamma, to_dev(rlk),
                            st if radices else None, d_dx=out["dx"], d_dgamma=out["dgamma"], d_dbeta=out["dbeta"])
    ref = orc.layernorm_grad(P, level, dy, xh, r, scale, scale, gamma, rlk, gal, keys)
    for k in shape:
        same(out[k], ref[k], k)


@pytest.mark.parametrize("part", ["dx", "dgamma", "dbeta"])
def test_layernorm_grad_single_parts(lib, orc, sets, part):
    """Each gradient alone; the weights' need fewer levels than the input's."""
    ctx, P = sets("small")
    level, B, F = {"dx": 5, "dgamma": 1, "dbeta": 0}[part], 2, 3
    announce("layernorm_grad %s alone" % part)
    st, (gal, keys) = steps(lib, P, [2], seed=6)
    dy, xh = words(P, 6, "dy", level + 1, (B, F, 2)), words(P, 6, "xh", level + 1, (B, F, 2))
    r, rlk = words(P, 6, "gr", level + 1, (B, 2)), key(P, 6, "rlk")
    shape = {"dx": (B, F, 2, level - 4, P.N), "dgamma": (F, 2, level, P.N), "dbeta": (F, 2, level + 1, P.N)}[part]
    out = empty_dev(shape)
    lib.ckks_layernorm_grad(ctx, to_dev(dy), B, F, level, to_dev(xh), level, 2.0 ** 37, to_dev(r), level, 2.0 ** 37, None,
                            to_dev(rlk), st, **{"d_" + part: out})
    same(out, orc.layernorm_grad(P, level, dy, xh, r, 2.0 ** 37, 2.0 ** 37, None, rlk, gal, keys, (part,))[part])
