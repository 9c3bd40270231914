"""Bit-exact parity of the attention calls (ckks_rotate_sum, ckks_attn_scores,
ckks_attn_mix, ckks_linattn_chunk, ckks_linattn_step) against the CPU oracle,
through the C interface: every output word must be equal, so there are no
tolerances.  Words are uniform residues (what encryption makes them), the top
of the residue range where lazy arithmetic comes closest to overflowing, or
real encryptions."""
import os
import subprocess
import sys

import numpy as np
import pytest

import ckks_synth as S
from gpu_util import announce, config_pair, empty_dev, make_pair, misaligned_dev, to_dev, to_host, torch_cuda
from helpers import encrypt_slots, galois_key, relin_key, secret

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# (log_n, L, q_bits, K, p_bits, dnum)
SETS = {
    "tiny": (12, 4, 30, 1, 60, 4),
    "small": (10, 6, 40, 2, 60, 3),
    "c3": (12, 24, 54, 8, 60, 3),
    "one_digit": (11, 12, 50, 12, 60, 1),
    "many_digits": (10, 9, 54, 1, 60, 9),
    "digit_each": (10, 14, 50, 1, 60, 14),  # 14 x 15 extended limbs: more transforms than one launch lists
    "q57": (13, 6, 57, 3, 60, 2),
    "mid": (13, 8, 54, 3, 60, 3),
    "mid14": (14, 5, 50, 2, 60, 3),
    "mid15": (15, 4, 45, 2, 60, 2),
    "mid57": (13, 6, 57, 3, 59, 2),
    "midwide": (13, 6, 62, 2, 61, 3),
    "mid16": (13, 16, 54, 16, 60, 1),
    "wide": (12, 6, 62, 2, 61, 3),
    "wide61": (11, 8, 61, 4, 62, 2),
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
    return fn(S.stream(seed, "attn/" + tag), P.q[:limbs], P.N, lead=lead)


def key(P, seed, tag, top=False):
    fn = S.top_limbs if top else S.uniform_limbs
    return fn(S.stream(seed, "attn/key/" + tag), P.mods, P.N, lead=(P.dnum, 2))


def steps(lib, P, radices, seed=0, top=False, stride=1):
    """(library stages, (galois, keys) for the oracle)."""
    gal, host = [], []
    for s, r in enumerate(radices):
        gal.append([P.galois(stride * k) for k in range(1, r)])
        host.append([key(P, seed, "%d.%d" % (s, k), top) for k in range(1, r)])
        stride = stride * r % (P.N // 2) or 1
    return lib.RotateSum(gal, [[to_dev(k) for k in ks] for ks in host]), (gal, host)


def same(got, ref, what=""):
    got = to_host(got)
    assert got.shape == ref.shape
    assert np.array_equal(got, ref), "%s: %d words differ" % (what, int((got != ref).sum()))


# ---------------------------------------------------------------- rotate_sum

SUMS = [
    ("tiny", 3, 1, [2]), ("tiny", 0, 3, [3, 2]), ("small", 5, 1, [4, 8]), ("small", 2, 9, [5]), ("small", 0, 2, [7]),
    ("c3", 23, 2, [8, 2]), ("c3", 16, 3, [3]), ("c3", 7, 1, [4]), ("one_digit", 11, 2, [6]), ("one_digit", 4, 1, [2, 2]),
    ("many_digits", 8, 2, [9]), ("many_digits", 3, 17, [2]), ("q57", 5, 3, [8]), ("wide", 5, 2, [8]), ("wide", 1, 1, [3]),
    ("wide61", 7, 2, [5, 3]), ("small", 3, 1, [32]), ("tiny", 2, 8, [4]),
    ("many_digits", 8, 1, [32]),  # 9 digits x 31 rotations: the column sums fold on the way
    ("many_digits", 8, 5, [32]),
    ("digit_each", 13, 2, [3]), ("small", 4, 131, [2]), ("c3", 23, 23, [2]),
    ("mid", 7, 2, [8]), ("mid14", 4, 5, [4, 2]), ("mid15", 3, 1, [3]), ("mid57", 5, 2, [4]), ("midwide", 5, 2, [3]),
    ("mid16", 15, 1, [3]),
]


@pytest.mark.parametrize("name,level,batch,radices", SUMS, ids=lambda v: str(v).replace(" ", ""))
def test_rotate_sum_parity(lib, orc, sets, name, level, batch, radices):
    ctx, P = sets(name)
    announce("rotate_sum %s level=%d batch=%d radices=%s" % (name, level, batch, radices))
    st, (gal, keys) = steps(lib, P, radices)
    x = words(P, level, "sum", level + 1, (batch, 2))
    out = empty_dev(x.shape)
    lib.ckks_rotate_sum(ctx, to_dev(x), out, batch, level, st)
    same(out, np.stack([orc.rotate_sum(P, level, c, gal, keys) for c in x]))


@pytest.mark.parametrize("name,level,radices", [("c3", 23, [8]), ("q57", 5, [32]), ("many_digits", 8, [32]),
                                                 ("wide", 5, [16]), ("wide61", 7, [8]), ("one_digit", 11, [8]),
                                                 ("mid", 7, [32]), ("midwide", 5, [8])])
@pytest.mark.parametrize("batch", [1, 2, 5])
def test_rotate_sum_top_of_range(lib, orc, sets, name, level, radices, batch):
    ctx, P = sets(name)
    announce("rotate_sum top of range %s batch=%d" % (name, batch))
    st, (gal, keys) = steps(lib, P, radices, top=True)
    x = words(P, 1, "top", level + 1, (batch, 2), top=True)
    x[0, 0, 0, :] = np.uint64(P.q[0] - 1)
    out = empty_dev(x.shape)
    lib.ckks_rotate_sum(ctx, to_dev(x), out, batch, level, st)
    same(out[0], orc.rotate_sum(P, level, x[0], gal, keys))
    same(out[batch - 1], orc.rotate_sum(P, level, x[batch - 1], gal, keys))


def test_rotate_sum_elements_twice_and_conjugation(lib, orc, sets):
    """The same element twice in a stage, and elements outside the powers of 5."""
    ctx, P = sets("small")
    announce("rotate_sum repeated elements")
    g = P.galois(3)
    gal = [[g, g, 2 * P.N - 1, 3]]
    host = [[key(P, 4, str(i)) for i in (0, 0, 1, 2)]]
    x = words(P, 4, "twice", 6, (1, 2))
    dev = [[to_dev(k) for k in host[0]]]
    dev[0][1] = dev[0][0]  # one key buffer, used twice
    out = empty_dev(x.shape)
    lib.ckks_rotate_sum(ctx, to_dev(x), out, 1, 5, lib.RotateSum(gal, dev))
    same(out[0], orc.rotate_sum(P, 5, x[0], gal, host))


def test_rotate_sum_encrypted(lib, orc, sets):
    """An encrypted vector summed over 16 slots at stride 4 decrypts to the sums (2^-12, as the tiny
    single-rotation set's other tests: 30-bit primes, scale 2^25)."""
    ctx, P = sets("tiny")
    announce("rotate_sum encrypted")
    s, s_ntt = secret(orc, P, 6, 64)
    gal = [[P.galois(4 * k) for k in range(1, 4)], [P.galois(16 * k) for k in range(1, 4)]]
    keys = [[to_dev(galois_key(orc, P, s_ntt, g, 6, "g%d" % g)) for g in gs] for gs in gal]
    z = S.uniform_slots(S.stream(6, "z"), P.N // 2)
    ct = encrypt_slots(orc, P, s_ntt, z, 2.0 ** 25, 3, 6, "ct")
    out = empty_dev((1,) + ct.shape)
    lib.ckks_rotate_sum(ctx, to_dev(ct[None]), out, 1, 3, lib.RotateSum(gal, keys))
    got = orc.decrypt(P, 3, to_host(out)[0], s_ntt, 2.0 ** 25)
    ref = sum(np.roll(z, -4 * k) for k in range(16))
    assert np.max(np.abs(got - ref)) / np.max(np.abs(ref)) < 2.0 ** -12


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("name,level,G,nq,nk,radices", [
    ("tiny", 3, 1, 1, 1, [2]), ("tiny", 1, 1, 2, 3, []), ("small", 5, 2, 3, 2, [4]), ("c3", 23, 1, 1, 2, [3]),
    ("c3", 12, 2, 1, 1, [2, 2]), ("wide", 5, 1, 2, 1, [3]), ("one_digit", 11, 1, 1, 1, [2]), ("small", 2, 1, 7, 5, [2]),
    ("mid", 7, 1, 2, 3, [4]), ("mid14", 1, 1, 1, 2, []), ("midwide", 3, 1, 1, 1, [2])])
def test_attn_scores_parity(lib, orc, sets, name, level, G, nq, nk, radices):
    ctx, P = sets(name)
    announce("attn_scores %s level=%d %dx%dx%d" % (name, level, G, nq, nk))
    st, ref_st = steps(lib, P, radices)
    q, k = words(P, level, "q", level + 1, (G, nq, 2)), words(P, level, "k", level + 1, (G, nk, 2))
    rlk = key(P, 0, "rlk")
    out = empty_dev((G, nq, nk, 2, level, P.N))
    lib.ckks_attn_scores(ctx, to_dev(q), nq, to_dev(k), nk, G, level, to_dev(rlk), st if radices else None, out)
    same(out, orc.attn_scores(P, level, q, k, rlk, *ref_st))


@pytest.mark.parametrize("name,level,G,nq,nk,M,radices", [
    ("tiny", 3, 1, 1, 1, 1, [2]), ("tiny", 2, 2, 2, 3, 1, []), ("tiny", 1, 1, 1, 2, 0, [2]), ("small", 5, 3, 2, 2, 2, [4]),
    ("small", 4, 2, 1, 9, 0, [2, 2]), ("c3", 12, 1, 2, 3, 1, [3]), ("wide", 5, 2, 1, 2, 2, [2]),
    ("wide61", 7, 1, 1, 9, 1, []), ("small", 3, 1, 11, 1, 1, [2]), ("mid", 7, 2, 2, 2, 2, [4]), ("mid14", 2, 1, 1, 2, 1, [2]),
    ("mid57", 5, 1, 1, 2, 0, []), ("midwide", 5, 1, 1, 2, 1, [2]), ("mid16", 15, 1, 1, 1, 1, [])])
@pytest.mark.parametrize("top", [False, True])
def test_attn_mix_parity(lib, orc, sets, name, level, G, nq, nk, M, radices, top):
    ctx, P = sets(name)
    announce("attn_mix %s level=%d %dx%dx%d mask=%d top=%d" % (name, level, G, nq, nk, M, top))
    st, ref_st = steps(lib, P, radices)
    a, v = words(P, level, "a", level + 1, (G, nq, nk, 2), top), words(P, level, "v", level + 1, (G, nk, 2), top)
    m = words(P, level, "m", level + 1, (M, nk), top) if M else None
    rlk = key(P, 0, "rlk", top)
    low = 2 if M else 1
    num, den = empty_dev((G, nq, 2, level + 1 - low, P.N)), empty_dev((G, nq, 2, level + 2 - low, P.N))
    args = (ctx, to_dev(a), nq, to_dev(v), nk, G, to_dev(m) if M else None, M, level, to_dev(rlk),
            st if radices else None)
    lib.ckks_attn_mix(*args, num, den)
    ref = orc.attn_mix(P, level, a, v, m, rlk, *ref_st)
    same(num, ref[0], "num")
    same(den, ref[1], "den")
    num.zero_()
    lib.ckks_attn_mix(*args, num)  # without the normaliser
    same(num, ref[0], "num alone")


def test_attn_mix_mask_that_leaves_nothing(lib, orc, sets):
    """A group whose mask rows are all zero: the trivial zero ciphertext through every step."""
    ctx, P = sets("small")
    announce("attn_mix empty group")
    a, v = words(P, 3, "ea", 6, (2, 1, 2, 2)), words(P, 3, "ev", 6, (2, 2, 2))
    m = words(P, 3, "em", 6, (2, 2))
    m[1] = 0
    st, ref_st = steps(lib, P, [4])
    rlk = key(P, 0, "rlk")
    num, den = empty_dev((2, 1, 2, 4, P.N)), empty_dev((2, 1, 2, 5, P.N))
    lib.ckks_attn_mix(ctx, to_dev(a), 1, to_dev(v), 2, 2, to_dev(m), 2, 5, to_dev(rlk), st, num, den)
    ref = orc.attn_mix(P, 5, a, v, m, rlk, *ref_st)
    same(num, ref[0])
    same(den, ref[1])
    assert not to_host(num)[1].any() and not to_host(den)[1].any()


CHUNKS = [
    # name, level, T, G, rows, read, carry, state, radices
    ("tiny", 3, 1, 1, 1, True, True, True, [2]), ("tiny", 3, 4, 1, 1, False, False, False, []),
    ("small", 5, 3, 2, 2, True, True, True, [4]), ("small", 5, 5, 3, 2, True, False, True, [2]),
    ("small", 4, 2, 2, 1, False, True, False, [2, 2]), ("c3", 23, 2, 1, 1, True, True, True, [3]),
    ("wide", 5, 3, 1, 1, True, True, True, [2]), ("wide61", 7, 2, 2, 1, True, False, False, [3]),
    ("one_digit", 11, 2, 1, 1, True, True, True, [2]), ("small", 3, 13, 1, 1, True, True, True, [2]),
    ("mid", 7, 2, 2, 1, True, True, True, [4]), ("mid14", 3, 2, 1, 1, False, False, True, [2]),
    ("mid15", 3, 1, 1, 1, True, True, False, []), ("mid57", 5, 2, 1, 1, True, False, True, [2]),
    ("midwide", 5, 3, 1, 1, True, True, True, [2]), ("mid16", 15, 1, 1, 1, False, False, True, [2]),
]


def chunk_case(P, level, T, G, R, read, carry, state, seed, top=False):
    d = {x: words(P, seed, x, level + 1, (T, G, 2), top) for x in "qkv"}
    d["w"] = words(P, seed, "w", level + 1, (T, R), top)
    d["r"] = words(P, seed, "r", level + 1, (T, R), top) if read else None
    d["carry"] = words(P, seed, "carry", level - 1, (R,), top) if carry else None
    d["state"] = words(P, seed, "state", level - 1, (G, 2), top) if state else None
    return d


def dev(x):
    return None if x is None else to_dev(x)


def run_chunk(lib, ctx, P, d, level, T, G, R, rlk, st):
    y = empty_dev((T, G, 2, level - 2, P.N))
    out = empty_dev((G, 2, level - 1 if d["carry"] is None else level - 2, P.N))
    lib.ckks_linattn_chunk(ctx, dev(d["q"]), dev(d["k"]), dev(d["v"]), T, G, dev(d["w"]), dev(d["r"]), dev(d["carry"]),
                           R, dev(d["state"]), level, to_dev(rlk), st, y, out)
    return y, out


@pytest.mark.parametrize("name,level,T,G,R,read,carry,state,radices", CHUNKS)
@pytest.mark.parametrize("top", [False, True])
def test_linattn_chunk_parity(lib, orc, sets, name, level, T, G, R, read, carry, state, radices, top):
    ctx, P = sets(name)
    announce("linattn_chunk %s level=%d T=%d G=%d R=%d read=%d carry=%d state=%d top=%d"
             % (name, level, T, G, R, read, carry, state, top))
    st, ref_st = steps(lib, P, radices)
    d = chunk_case(P, level, T, G, R, read, carry, state, level + T, top)
    d["w"][-1, 0] = 0  # a padded token
    rlk = key(P, 0, "rlk", top)
    y, out = run_chunk(lib, ctx, P, d, level, T, G, R, rlk, st if radices else None)
    ref = orc.linattn_chunk(P, level, d["q"], d["k"], d["v"], d["w"], d["r"], d["carry"], d["state"], rlk, *ref_st)
    same(y, ref[0], "y")
    same(out, ref[1], "state")


@pytest.mark.parametrize("name,level,G,R,state,radices", [
    ("tiny", 3, 1, 1, True, [2]), ("tiny", 2, 1, 0, True, [3]), ("tiny", 3, 2, 1, False, []), ("small", 5, 3, 2, True, [4]),
    ("small", 4, 11, 11, True, [2]), ("small", 2, 2, 0, False, [2, 2]), ("c3", 23, 2, 1, True, [3]),
    ("c3", 12, 1, 0, True, [8]), ("wide", 5, 2, 1, True, [2]), ("wide61", 7, 1, 0, True, [2]),
    ("many_digits", 8, 1, 1, True, [2]), ("one_digit", 6, 1, 1, True, [2]), ("digit_each", 13, 1, 1, True, [2]),
    ("mid", 7, 3, 2, True, [4]), ("mid14", 2, 1, 0, True, []), ("mid15", 3, 1, 1, True, [2]), ("mid57", 5, 2, 0, True, [2]),
    ("midwide", 5, 2, 1, True, [2]), ("mid16", 15, 1, 1, True, [])])
@pytest.mark.parametrize("top", [False, True])
def test_linattn_step_parity(lib, orc, sets, name, level, G, R, state, radices, top):
    ctx, P = sets(name)
    announce("linattn_step %s level=%d G=%d R=%d state=%d top=%d" % (name, level, G, R, state, top))
    st, ref_st = steps(lib, P, radices)
    q, k, v = (words(P, level, x, level + 1, (G, 2), top) for x in "qkv")
    dec = words(P, level, "dec", level + 1, (R,), top) if R else None
    s_in = words(P, level, "st", level + (1 if R else 0), (G, 2), top) if state else None
    rlk = key(P, 0, "rlk", top)
    y, out = empty_dev((G, 2, level - 1, P.N)), empty_dev((G, 2, level, P.N))
    lib.ckks_linattn_step(ctx, to_dev(q), to_dev(k), to_dev(v), G, dev(dec), R, dev(s_in), level, to_dev(rlk),
                          st if radices else None, y, out)
    ref = orc.linattn_step(P, level, q, k, v, dec, s_in, rlk, *ref_st)
    same(y, ref[0], "y")
    same(out, ref[1], "state")


def test_prompt_then_tokens_then_cross_attention(lib, orc, sets):
    """The calls as a decoder layer runs them: a prompt's chunk, single tokens on its state, scores of the
    outputs against an encoder's keys, the polynomial weights, the mix; one stream, nothing in between."""
    ctx, P = sets("c3")
    announce("prompt, tokens, cross attention")
    st, ref_st = steps(lib, P, [4])
    rlk = key(P, 0, "rlk")
    d_rlk = to_dev(rlk)
    T, G, R, lv = 3, 2, 1, 23
    d = chunk_case(P, lv, T, G, R, True, True, True, 77)
    y, state = run_chunk(lib, ctx, P, d, lv, T, G, R, rlk, st)
    ref_y, ref_s = orc.linattn_chunk(P, lv, d["q"], d["k"], d["v"], d["w"], d["r"], d["carry"], d["state"], rlk, *ref_st)
    lv = 20
    for i in range(2):
        q, k, v = (words(P, 80 + i, x, lv + 1, (G, 2)) for x in "qkv")
        dec = words(P, 80 + i, "dec", lv + 1, (R,))
        ny, ns = empty_dev((G, 2, lv - 1, P.N)), empty_dev((G, 2, lv, P.N))
        lib.ckks_linattn_step(ctx, to_dev(q), to_dev(k), to_dev(v), G, to_dev(dec), R, state, lv, d_rlk, st, ny, ns)
        ref_ny, ref_s = orc.linattn_step(P, lv, q, k, v, dec, ref_s, rlk, *ref_st)
        state, lv = ns, lv - 1
    lq = lv - 1  # the last step's output level
    keys_ = words(P, 90, "ek", lq + 1, (G, 2, 2))
    vals = words(P, 90, "ev", lq - 2, (G, 2, 2))
    s = empty_dev((G, 1, 2, 2, lq, P.N))
    lib.ckks_attn_scores(ctx, ny, 1, to_dev(keys_), 2, G, lq, d_rlk, st, s)
    ref_sc = orc.attn_scores(P, lq, ref_ny[:, None], keys_, rlk, *ref_st)
    p = empty_dev((G * 2, 2, lq - 2, P.N))
    lib.ckks_poly_eval_tree(ctx, s, G * 2, lq - 1, 2.0 ** 54, [1.0, 1.0, 0.5], d_rlk, p)
    ref_p, _ = orc.poly_eval_tree(P, lq - 1, ref_sc.reshape((-1,) + ref_sc.shape[3:]), 2.0 ** 54, [1.0, 1.0, 0.5], rlk)
    la = lq - 3
    mask = words(P, 90, "em", la + 1, (1, 2))
    num, den = empty_dev((G, 1, 2, la - 1, P.N)), empty_dev((G, 1, 2, la, P.N))
    lib.ckks_attn_mix(ctx, p, 1, to_dev(vals), 2, G, to_dev(mask), 1, la, d_rlk, st, num, den)
    ref = orc.attn_mix(P, la, ref_p.reshape((G, 1, 2) + ref_p.shape[1:]), vals, mask, rlk, *ref_st)
    same(y, ref_y)
    same(num, ref[0])
    same(den, ref[1])


# ---------------------------------------------------------------- use

def test_bytes_outside_the_outputs_stay(lib, orc, sets):
    """Outputs inside a larger buffer: the words before and behind them are left as they were."""
    torch = torch_cuda()
    ctx, P = sets("small")
    announce("guard words")
    st, _ = steps(lib, P, [3])
    rlk = to_dev(key(P, 0, "rlk"))
    lv, G, N = 5, 3, P.N
    q, k, v = (to_dev(words(P, 1, x, lv + 1, (2, G, 2))) for x in "qkv")
    w = to_dev(words(P, 1, "w", lv + 1, (2, 1)))
    ny, ns = 2 * G * 2 * (lv - 2) * N, G * 2 * (lv - 1) * N
    buf = torch.full((ny + ns + 6 * N,), -7, dtype=torch.int64, device="cuda")
    y, s = buf[2 * N:2 * N + ny], buf[4 * N + ny:4 * N + ny + ns]
    lib.ckks_linattn_chunk(ctx, q, k, v, 2, G, w, None, None, 1, None, lv, rlk, st, y, s)
    h = to_host(buf).view(np.int64)
    for part in (h[:2 * N], h[2 * N + ny:4 * N + ny], h[4 * N + ny + ns:]):
        assert (part == -7).all()
    assert (h[2 * N:2 * N + ny] != -7).all() and (h[4 * N + ny:4 * N + ny + ns] != -7).all()


def test_blocks_of_items_and_tokens(lib, orc, sets):
    """More tokens, groups and items than one launch of a stage takes; repeated calls give the same words."""
    torch = torch_cuda()
    ctx, P = sets("small")
    announce("many items")
    st, ref_st = steps(lib, P, [2])
    rlk = key(P, 0, "rlk")
    T, G = 21, 2
    d = chunk_case(P, 3, T, G, 1, True, False, True, 5)
    y, out = run_chunk(lib, ctx, P, d, 3, T, G, 1, rlk, st)
    first = y.clone()
    ref = orc.linattn_chunk(P, 3, d["q"], d["k"], d["v"], d["w"], d["r"], None, d["state"], rlk, *ref_st)
    same(y, ref[0])
    same(out, ref[1])
    y2, _ = run_chunk(lib, ctx, P, d, 3, T, G, 1, rlk, st)
    assert torch.equal(first, y2)


def test_chunk_of_more_items_than_a_launch(lib, orc, sets):
    """66 tokens of 2 groups with read weights and a carry, each group its own rows: products, rescales and
    relinearisations go in several launches."""
    ctx, P = sets("small")
    announce("chunk of 132 items")
    st, ref_st = steps(lib, P, [2])
    rlk = key(P, 0, "rlk")
    T, G = 66, 2
    d = chunk_case(P, 3, T, G, 2, True, True, True, 6)
    y, out = run_chunk(lib, ctx, P, d, 3, T, G, 2, rlk, st)
    ref = orc.linattn_chunk(P, 3, d["q"], d["k"], d["v"], d["w"], d["r"], d["carry"], d["state"], rlk, *ref_st)
    same(y, ref[0])
    same(out, ref[1])


def test_small_blocks(lib, orc, sets, monkeypatch):
    """Intermediates limited to 1 MiB: every call runs in blocks of one or two items, a chunk's tokens in
    several blocks that carry the prefix sums, its groups in several blocks whose outputs interleave."""
    monkeypatch.setenv("CKKS_BLOCK_MB", "1")
    ctx, P = sets("small")
    announce("small blocks")
    st, ref_st = steps(lib, P, [2])
    rlk = key(P, 0, "rlk")
    d_rlk = to_dev(rlk)
    for T, G, R in [(5, 1, 1), (4, 5, 2), (40, 1, 1)]:
        d = chunk_case(P, 5, T, G, R, T < 6, False, True, 30 + T)
        y, out = run_chunk(lib, ctx, P, d, 5, T, G, R, rlk, st)
        ref = orc.linattn_chunk(P, 5, d["q"], d["k"], d["v"], d["w"], d["r"], None, d["state"], rlk, *ref_st)
        same(y, ref[0], "y %d %d" % (T, G))
        same(out, ref[1], "state %d %d" % (T, G))
    a, v, m = words(P, 8, "a", 6, (2, 3, 2, 2)), words(P, 8, "v", 6, (2, 2, 2)), words(P, 8, "m", 6, (2, 2))
    num, den = empty_dev((2, 3, 2, 4, P.N)), empty_dev((2, 3, 2, 5, P.N))
    lib.ckks_attn_mix(ctx, to_dev(a), 3, to_dev(v), 2, 2, to_dev(m), 2, 5, d_rlk, st, num, den)
    ref = orc.attn_mix(P, 5, a, v, m, rlk, *ref_st)
    same(num, ref[0])
    same(den, ref[1])
    s = empty_dev((2, 3, 2, 2, 5, P.N))
    lib.ckks_attn_scores(ctx, to_dev(a[:, :, 0]), 3, to_dev(v), 2, 2, 5, d_rlk, st, s)
    same(s, orc.attn_scores(P, 5, a[:, :, 0], v, rlk, *ref_st))
    q, k, w = (words(P, 9, x, 6, (7, 2)) for x in "qkv")
    for R in (0, 3):
        dec, s_in = (words(P, 9, "dec", 6, (R,)), words(P, 9, "st", 6, (7, 2))) if R else (None, words(P, 9, "st", 5, (7, 2)))
        y, out = empty_dev((7, 2, 4, P.N)), empty_dev((7, 2, 5, P.N))
        lib.ckks_linattn_step(ctx, to_dev(q), to_dev(k), to_dev(w), 7, dev(dec), R, to_dev(s_in), 5, d_rlk, st, y, out)
        ref = orc.linattn_step(P, 5, q, k, w, dec, s_in, rlk, *ref_st)
        same(y, ref[0])
        same(out, ref[1])


def test_on_another_stream(lib, orc, sets):
    """A side stream, while the default stream is busy: the call waits for nothing but its own stream."""
    torch = torch_cuda()
    ctx, P = sets("small")
    announce("side stream")
    st, (gal, keys) = steps(lib, P, [4])
    x = words(P, 2, "stream", 6, (2, 2))
    dx, out = to_dev(x), empty_dev(x.shape)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        lib.ckks_rotate_sum(ctx, dx, out, 2, 5, st)  # the current stream
    side.synchronize()
    ref = np.stack([orc.rotate_sum(P, 5, c, gal, keys) for c in x])
    same(out, ref)
    out.zero_()
    torch.cuda.synchronize()
    lib.ckks_rotate_sum(ctx, dx, out, 2, 5, st, stream=side)
    side.synchronize()
    same(out, ref)


def test_two_contexts_on_two_streams(lib, orc, sets):
    """Calls of two contexts in flight at once on two streams."""
    torch = torch_cuda()
    made = [sets("mid"), make_pair(lib, orc, *SETS["small"])]
    announce("two contexts")
    runs = []
    for n, (ctx, P) in enumerate(made):
        st, ref_st = steps(lib, P, [4, 2], seed=n)
        x = words(P, n, "two", P.L, (6, 2))
        runs.append((ctx, P, st, ref_st, x, to_dev(x), empty_dev(x.shape), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for ctx, P, st, _, x, dx, out, stream in runs:
            lib.ckks_rotate_sum(ctx, dx, out, 6, P.L - 1, st, stream=stream)
    torch.cuda.synchronize()
    for ctx, P, st, ref_st, x, dx, out, stream in runs:
        same(out[0], orc.rotate_sum(P, P.L - 1, x[0], *ref_st))
        same(out[5], orc.rotate_sum(P, P.L - 1, x[5], *ref_st))
    made[1][0].close()


def test_calls_in_a_row_without_waiting(lib, orc, sets):
    """Mixes and chunks on one stream with nothing waited for between them: the steps on the internal stream
    start after the call before has finished with the context's buffers."""
    torch = torch_cuda()
    ctx, P = sets("mid")
    announce("calls in a row")
    st, ref_st = steps(lib, P, [2])
    rlk = key(P, 0, "rlk")
    d_rlk = to_dev(rlk)
    lv, n, made = 5, 6, []
    for i in range(4):
        c = {t: words(P, i, "row" + t, n, (2, 1, 2)) for t in "avqkx"}
        p = {t: words(P, i, "row" + t, n, (2, 1)) for t in "mwr"}
        car, s_in = words(P, i, "rowc", n - 2, (1,)), words(P, i, "rows", n - 2, (1, 2))
        made.append((c, p, car, s_in, {t: to_dev(x) for t, x in {**c, **p}.items()}, to_dev(car), to_dev(s_in),
                     empty_dev((1, 2, lv - 1, P.N)), empty_dev((1, 2, lv, P.N)), empty_dev((2, 1, 2, lv - 2, P.N)),
                     empty_dev((1, 2, lv - 2, P.N))))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for c, p, car, s_in, d, d_car, d_s, num, den, y, end in made:
            lib.ckks_attn_mix(ctx, d["a"], 1, d["v"], 2, 1, d["m"], 1, lv, d_rlk, st, num, den)
            lib.ckks_linattn_chunk(ctx, d["q"], d["k"], d["x"], 2, 1, d["w"], d["r"], d_car, 1, d_s, lv, d_rlk, st, y,
                                   end)
    side.synchronize()
    for i, (c, p, car, s_in, d, d_car, d_s, num, den, y, end) in enumerate(made):
        rn, rd = orc.attn_mix(P, lv, c["a"][None, None, :, 0], c["v"][None, :, 0], p["m"][None, :, 0], rlk, *ref_st)
        same(num, rn[0], "num %d" % i)
        same(den, rd[0], "den %d" % i)
        ry, rs = orc.linattn_chunk(P, lv, c["q"], c["k"], c["x"], p["w"], p["r"], car, s_in, rlk, *ref_st)
        same(y, ry, "y %d" % i)
        same(end, rs, "state %d" % i)


def test_one_buffer_as_several_operands(lib, orc, sets):
    """Inputs may be one another: self-products, and one key as the relinearisation's and a rotation's."""
    ctx, P = sets("small")
    announce("one buffer as several operands")
    gal, host = [[P.galois(1)]], [[key(P, 3, "both")]]
    d_key = to_dev(host[0][0])
    st = lib.RotateSum(gal, [[d_key]])
    x = words(P, 3, "self", 6, (2, 2))
    dx = to_dev(x)
    out = empty_dev((1, 2, 2, 2, 5, P.N))
    lib.ckks_attn_scores(ctx, dx, 2, dx, 2, 1, 5, d_key, st, out)
    same(out, orc.attn_scores(P, 5, x[None], x[None], host[0][0], gal, host))
    y, s_out = empty_dev((2, 2, 4, P.N)), empty_dev((2, 2, 5, P.N))
    pt = words(P, 3, "selfpt", 6, (1,))
    lib.ckks_linattn_step(ctx, dx, dx, dx, 2, to_dev(pt), 1, dx, 5, d_key, st, y, s_out)
    ref = orc.linattn_step(P, 5, x, x, x, pt, x, host[0][0], gal, host)
    same(y, ref[0])
    same(s_out, ref[1])


def test_traced_families(lib, orc, sets):
    """The families of the attention kernels count their launches, on the internal stream too."""
    ctx, P = sets("mid")
    announce("traced families")
    st, _ = steps(lib, P, [2, 2])
    rlk = to_dev(key(P, 0, "rlk"))
    a, v = to_dev(words(P, 1, "ta", 4, (1, 2))), to_dev(words(P, 1, "tv", 4, (1, 2)))
    num, den = empty_dev((1, 2, 3, P.N)), empty_dev((1, 2, 4, P.N))
    counts = {}
    for family in ("sum_ip", "attn_mac"):
        lib.ckks_trace_begin(ctx, family)
        lib.ckks_attn_mix(ctx, a, 1, v, 1, 1, None, 0, 3, rlk, st, num, den)
        t = lib.ckks_trace_end(ctx)
        counts[family] = t["launches"]
        assert t["work_units"] > 0
    assert counts == {"sum_ip": 4, "attn_mac": 1}


def test_captured_step_replays(lib, orc):
    """A step captured into a graph after one eager call: every replay equals the eager words, with new
    inputs, with eager work of the same context between the replays, and after a larger call has grown the
    context's buffers."""
    torch = torch_cuda()
    ctx, P = make_pair(lib, orc, *SETS["small"])
    announce("captured step")
    st, ref_st = steps(lib, P, [2, 2])
    rlk = key(P, 0, "rlk")
    d_rlk = to_dev(rlk)
    lv, G = 5, 6  # two chunks of the relinearisation: the internal streams join the capture

    def inputs(seed):
        return [words(P, seed, x, lv + 1, (G, 2)) for x in "qkv"] + [words(P, seed, "dec", lv + 1, (1,)),
                                                                     words(P, seed, "st", lv + 1, (G, 2))]

    bufs = [to_dev(x) for x in inputs(0)]
    y, out = empty_dev((G, 2, lv - 1, P.N)), empty_dev((G, 2, lv, P.N))

    def call():
        lib.ckks_linattn_step(ctx, bufs[0], bufs[1], bufs[2], G, bufs[3], 1, bufs[4], lv, d_rlk, st, y, out)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call()  # sizes the context's buffers
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call()
    for i in range(4):
        host = inputs(10 + i)
        for b, h in zip(bufs, host):
            b.copy_(to_dev(h))
        y.zero_()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        q, k, v, dec, s_in = host
        ref = orc.linattn_step(P, lv, q, k, v, dec, s_in, rlk, *ref_st)
        same(y, ref[0], "replay %d" % i)
        same(out, ref[1], "replay %d" % i)
        if i == 1:  # a larger eager call grows the buffers the graph was captured on
            big = words(P, 50, "big", 6, (40, 2))
            o = empty_dev(big.shape)
            lib.ckks_rotate_sum(ctx, to_dev(big), o, 40, 5, st)
            same(o[39], orc.rotate_sum(P, 5, big[39], *ref_st))
        call()
        torch.cuda.synchronize()
        same(y, ref[0], "eager after replay %d" % i)
    del graph
    ctx.close()


def test_capture_of_a_first_call_is_refused(lib, orc):
    """A call that would have to grow the context's buffers during a capture raises and leaves the capture
    usable."""
    torch = torch_cuda()
    ctx, P = make_pair(lib, orc, *SETS["small"])
    announce("capture without a first call")
    st, _ = steps(lib, P, [2])
    x, out = to_dev(words(P, 2, "cap", 6, (1, 2))), empty_dev((1, 2, 6, P.N))
    marker = torch.zeros(8, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        with pytest.raises(lib.CKKSError) as e:
            lib.ckks_rotate_sum(ctx, x, out, 1, 5, st)
        marker.add_(1.0)
    assert e.value.code == lib.CKKS_EHIP and "captured" in str(e.value)
    graph.replay()
    torch.cuda.synchronize()
    assert marker.tolist() == [1.0] * 8
    lib.ckks_rotate_sum(ctx, x, out, 1, 5, st)
    torch.cuda.synchronize()
    ctx.close()


def test_captured_mix_and_chunk_replay(lib, orc):
    """The calls that run steps side by side on an internal stream, captured: every replay equals the oracle's
    words for its inputs, with eager calls of the same context between the replays."""
    torch = torch_cuda()
    ctx, P = make_pair(lib, orc, *SETS["small"])
    announce("captured mix and chunk")
    st, ref_st = steps(lib, P, [3])
    rlk = key(P, 0, "rlk")
    d_rlk = to_dev(rlk)
    lv, n = 5, 6
    names = ("a", "v", "q", "k", "x")

    def inputs(seed):
        return ({t: words(P, seed, t, n, (2, 2)) for t in names}, {t: words(P, seed, t, n, (2,)) for t in ("m", "w", "r")},
                words(P, seed, "carry", n - 2, (1,)), words(P, seed, "s", n - 2, (1, 2)))

    host = inputs(0)
    ct, pt = ({t: to_dev(x) for t, x in h.items()} for h in host[:2])
    carry, state = to_dev(host[2]), to_dev(host[3])
    num, den = empty_dev((1, 2, lv - 1, P.N)), empty_dev((1, 2, lv, P.N))
    y, end = empty_dev((2, 2, lv - 2, P.N)), empty_dev((1, 2, lv - 2, P.N))

    def call():
        lib.ckks_attn_mix(ctx, ct["a"], 1, ct["v"], 2, 1, pt["m"], 1, lv, d_rlk, st, num, den)
        lib.ckks_linattn_chunk(ctx, ct["q"], ct["k"], ct["x"], 2, 1, pt["w"], pt["r"], carry, 1, state, lv, d_rlk, st,
                               y, end)

    def check(h, what):
        c, p, car, s_in = h
        rn, rd = orc.attn_mix(P, lv, c["a"][None, None], c["v"][None], p["m"][None], rlk, *ref_st)
        same(num, rn[0], what)
        same(den, rd[0], what)
        ry, rs = orc.linattn_chunk(P, lv, c["q"][:, None], c["k"][:, None], c["x"][:, None], p["w"][:, None],
                                   p["r"][:, None], car, s_in, rlk, *ref_st)
        same(y, ry[:, 0], what)
        same(end, rs, what)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call()
    for i in range(4):
        host = inputs(10 + i)
        for group, h in zip((ct, pt), host):
            for t, x in h.items():
                group[t].copy_(to_dev(x))
        carry.copy_(to_dev(host[2]))
        state.copy_(to_dev(host[3]))
        for o in (num, den, y, end):
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(host, "replay %d" % i)
        for o in (num, den, y, end):
            o.zero_()
        call()
        torch.cuda.synchronize()
        check(host, "eager after replay %d" % i)
    del graph
    ctx.close()


def test_capture_before_the_internal_streams_is_refused(lib, orc):
    """A call that would create the internal streams during a capture raises, though the buffers are large enough."""
    torch = torch_cuda()
    ctx, P = make_pair(lib, orc, *SETS["small"])
    announce("capture without internal streams")
    st, ref_st = steps(lib, P, [2])
    rlk = key(P, 0, "rlk")
    d_rlk = to_dev(rlk)
    a, v = (words(P, 1, t, 6, (8, 2)) for t in "av")
    da, dv = to_dev(a), to_dev(v)
    num, den = empty_dev((8, 2, 5, P.N)), empty_dev((8, 2, 6, P.N))
    lib.ckks_attn_mix(ctx, da, 1, dv, 1, 8, None, 0, 5, d_rlk, st, num, None)  # no normaliser: one stream
    torch.cuda.synchronize()
    marker = torch.zeros(8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        with pytest.raises(lib.CKKSError) as e:
            lib.ckks_attn_mix(ctx, da, 1, dv, 1, 1, None, 0, 5, d_rlk, st, num, den)
        marker.add_(1.0)
    assert e.value.code == lib.CKKS_EHIP and "captured" in str(e.value)
    graph.replay()
    torch.cuda.synchronize()
    assert marker.tolist() == [1.0] * 8
    lib.ckks_attn_mix(ctx, da, 1, dv, 1, 1, None, 0, 5, d_rlk, st, num, den)
    torch.cuda.synchronize()
    rn, rd = orc.attn_mix(P, 5, a[:1, None, None], v[:1, None], None, rlk, *ref_st)
    same(num[:1], rn[0])
    same(den[:1], rd[0])
    ctx.close()


# ---------------------------------------------------------------- refusals

def refused(lib, code, fn, text=None):
    with pytest.raises(lib.CKKSError) as e:
        fn()
    assert e.value.code == code, str(e.value)
    if text:
        assert text in str(e.value)


def test_refusals(lib, orc, sets):
    torch = torch_cuda()
    ctx, P = sets("tiny")
    announce("refusals")
    N = P.N
    st, _ = steps(lib, P, [2])
    rlk = to_dev(key(P, 0, "rlk"))
    x = to_dev(words(P, 1, "x", 4, (2, 2)))
    pt = to_dev(words(P, 1, "pt", 4, (2,)))
    out = torch.full((2, 2, 4, N), 5, dtype=torch.int64, device="cuda")
    out2 = torch.full((2, 2, 4, N), 5, dtype=torch.int64, device="cuda")
    k1 = st.keys[0]

    def rs(steps_, batch=1, level=3, o=out, i=x):
        return lambda: lib.ckks_rotate_sum(ctx, i, o, batch, level, steps_)

    refused(lib, lib.CKKS_EINVAL, rs(lib.RotateSum([], [])), "at least one stage")
    refused(lib, lib.CKKS_EINVAL, rs(None), "at least one stage")
    refused(lib, lib.CKKS_EINVAL, rs(lib.RotateSum([[]], [[]])), "radix")
    refused(lib, lib.CKKS_EINVAL, rs(lib.RotateSum([[5] * 32], [[k1] * 32])), "radix")
    refused(lib, lib.CKKS_EINVAL, rs(lib.RotateSum([[5]] * 17, [[k1]] * 17)), "number of sum stages")
    refused(lib, lib.CKKS_EINVAL, rs(lib.RotateSum([[4]], [[k1]])), "odd")
    refused(lib, lib.CKKS_EINVAL, rs(lib.RotateSum([[2 * N + 1]], [[k1]])), "odd")
    refused(lib, lib.CKKS_EINVAL, rs(lib.RotateSum([[1]], [[k1]])), "identity")
    refused(lib, lib.CKKS_ERANGE, rs(st, level=4))
    refused(lib, lib.CKKS_ERANGE, rs(st, level=-1))
    refused(lib, lib.CKKS_EINVAL, rs(st, batch=-1))
    refused(lib, lib.CKKS_EINVAL, rs(st, o=x), "overlaps")
    refused(lib, lib.CKKS_EINVAL, rs(st, o=k1.view(-1)[: 2 * 4 * N]), "overlaps")
    mis = misaligned_dev((1, 2, 4, N))
    refused(lib, lib.CKKS_EINVAL, rs(st, o=mis), "aligned")
    refused(lib, lib.CKKS_EINVAL, rs(lib.RotateSum([[5]], [[misaligned_dev(tuple(k1.shape))]])), "aligned")
    with pytest.raises(lib.ArgumentError):
        rs(lib.RotateSum([[5]], [[None]]))()
    with pytest.raises(lib.ArgumentError):
        rs(st, batch=3)()
    with pytest.raises(lib.ArgumentError):
        rs(lib.RotateSum([[5]], [[x]]))()  # too short for a key

    sc = lambda nq=1, nk=1, G=1, lv=3, o=out, r=rlk: lambda: lib.ckks_attn_scores(ctx, x, nq, x, nk, G, lv, r, st, o)
    refused(lib, lib.CKKS_ERANGE, sc(lv=0))
    refused(lib, lib.CKKS_ERANGE, sc(lv=9))
    refused(lib, lib.CKKS_EINVAL, sc(nq=-1))
    refused(lib, lib.CKKS_EINVAL, sc(o=x), "overlaps")
    rc = lib.lib().ckks_attn_scores(ctx.handle, x.data_ptr(), 5000, x.data_ptr(), 0, 5000, 3, rlk.data_ptr(), None,
                                    out.data_ptr(), None)
    assert rc == lib.CKKS_EINVAL and "too many" in lib.ckks_last_error()

    def mx(nq=1, nk=1, G=1, m=pt, M=1, lv=3, o=out, e=out2):
        return lambda: lib.ckks_attn_mix(ctx, x, nq, x, nk, G, m, M, lv, rlk, st, o, e)

    refused(lib, lib.CKKS_EINVAL, mx(nk=0))
    refused(lib, lib.CKKS_EINVAL, mx(M=0), "mask")
    refused(lib, lib.CKKS_EINVAL, mx(M=2), "mask")
    refused(lib, lib.CKKS_EINVAL, mx(m=None, M=1), "mask")
    refused(lib, lib.CKKS_ERANGE, mx(lv=1))
    refused(lib, lib.CKKS_ERANGE, mx(m=None, M=0, lv=0))
    refused(lib, lib.CKKS_EINVAL, mx(e=out), "overlaps")
    refused(lib, lib.CKKS_EINVAL, mx(o=x), "overlaps")

    def ch(T=1, G=1, R=1, lv=3, o=out, so=out2, carry=None, state=None):
        return lambda: lib.ckks_linattn_chunk(ctx, x, x, x, T, G, pt, None, carry, R, state, lv, rlk, st, o, so)

    refused(lib, lib.CKKS_EINVAL, ch(T=0))
    refused(lib, lib.CKKS_EINVAL, ch(G=-1))
    refused(lib, lib.CKKS_EINVAL, ch(R=0), "rows")
    refused(lib, lib.CKKS_EINVAL, ch(R=2), "rows")
    refused(lib, lib.CKKS_ERANGE, ch(lv=2))
    refused(lib, lib.CKKS_EINVAL, ch(so=out), "overlaps")
    refused(lib, lib.CKKS_EINVAL, ch(state=out2), "overlaps")

    def sp(G=1, dec=pt, R=1, state=None, lv=3, o=out, so=out2):
        return lambda: lib.ckks_linattn_step(ctx, x, x, x, G, dec, R, state, lv, rlk, st, o, so)

    refused(lib, lib.CKKS_EINVAL, sp(R=0), "rows")
    refused(lib, lib.CKKS_EINVAL, sp(dec=None, R=1), "rows")
    refused(lib, lib.CKKS_EINVAL, sp(G=-2))
    refused(lib, lib.CKKS_ERANGE, sp(lv=1))
    refused(lib, lib.CKKS_EINVAL, sp(state=out2), "overlaps")
    with pytest.raises(lib.ArgumentError):
        sp(G=2, R=2, lv=3, o=out.view(-1)[: 8 * N - 2])()
    torch.cuda.synchronize()
    assert (out == 5).all() and (out2 == 5).all()  # a refused call writes nothing


def test_no_special_primes_is_refused(lib, orc):
    announce("no special primes")
    q = lib.ckks_find_primes(10, 40, 4)
    ctx = lib.Context(10, q, [], 2)
    x = to_dev(np.zeros((1, 2, 4, 1024), dtype=np.uint64))
    k = to_dev(np.zeros((2, 2, 4, 1024), dtype=np.uint64))
    st = lib.RotateSum([[5]], [[k]])
    o, o2 = empty_dev((1, 2, 4, 1024)), empty_dev((1, 2, 4, 1024))
    pt = to_dev(np.zeros((1, 4, 1024), dtype=np.uint64))
    refused(lib, lib.CKKS_EPARAM, lambda: lib.ckks_rotate_sum(ctx, x, o, 1, 3, st))
    refused(lib, lib.CKKS_EPARAM, lambda: lib.ckks_attn_scores(ctx, x, 1, x, 1, 1, 3, k, st, o))
    refused(lib, lib.CKKS_EPARAM, lambda: lib.ckks_attn_mix(ctx, x, 1, x, 1, 1, None, 0, 3, k, st, o))
    refused(lib, lib.CKKS_EPARAM, lambda: lib.ckks_linattn_chunk(ctx, x, x, x, 1, 1, pt, None, None, 1, None, 3, k, st, o,
                                                                 o2))
    refused(lib, lib.CKKS_EPARAM, lambda: lib.ckks_linattn_step(ctx, x, x, x, 1, None, 0, None, 3, k, st, o, o2))
    ctx.close()


def test_nothing_to_do(lib, orc, sets):
    ctx, P = sets("tiny")
    announce("empty calls")
    st, _ = steps(lib, P, [2])
    rlk = to_dev(key(P, 0, "rlk"))
    x, pt = to_dev(words(P, 1, "x", 4, (1, 2))), to_dev(words(P, 1, "pt", 4, (1,)))
    torch = torch_cuda()
    o, o2 = (torch.full((1, 2, 4, P.N), 5, dtype=torch.int64, device="cuda") for _ in range(2))
    lib.ckks_rotate_sum(ctx, x, o, 0, 3, st)
    lib.ckks_attn_scores(ctx, x, 0, x, 1, 1, 3, rlk, st, o)
    lib.ckks_attn_scores(ctx, x, 1, x, 0, 1, 3, rlk, st, o)
    lib.ckks_attn_mix(ctx, x, 0, x, 1, 1, pt, 1, 3, rlk, st, o, o2)
    lib.ckks_linattn_chunk(ctx, x, x, x, 1, 0, pt, None, None, 1, None, 3, rlk, st, o, o2)
    lib.ckks_linattn_step(ctx, x, x, x, 0, pt, 1, None, 3, rlk, st, o, o2)
    torch.cuda.synchronize()
    assert (o == 5).all() and (o2 == 5).all()


@pytest.mark.parametrize("op", ["sum", "step"])
def test_full_size(lib, orc, op):
    """N = 2^16, 24 + 8 primes at the top level: one ciphertext against the oracle, word for word."""
    ctx, P = config_pair(lib, orc, "C3")
    announce("full size %s" % op)
    st, ref_st = steps(lib, P, [3])
    if op == "sum":
        x = words(P, 1, "full", 24, (1, 2))
        out = empty_dev(x.shape)
        lib.ckks_rotate_sum(ctx, to_dev(x), out, 1, 23, st)
        same(out[0], orc.rotate_sum(P, 23, x[0], *ref_st))
    else:
        q, k, v, s_in = (words(P, 1, t, 13, (1, 2)) for t in ("q", "k", "v", "s"))
        dec, rlk = words(P, 1, "dec", 13, (1,)), key(P, 0, "rlk")
        y, out = empty_dev((1, 2, 11, P.N)), empty_dev((1, 2, 12, P.N))
        lib.ckks_linattn_step(ctx, to_dev(q), to_dev(k), to_dev(v), 1, to_dev(dec), 1, to_dev(s_in), 12, to_dev(rlk), st,
                              y, out)
        ref = orc.linattn_step(P, 12, q, k, v, dec, s_in, rlk, *ref_st)
        same(y, ref[0])
        same(out, ref[1])
    ctx.close()


# ---------------------------------------------------------------- forms that the cases above do not reach

SETS["q57low"] = (10, 6, 57, 3, 60, 2)


@pytest.mark.parametrize("name,level,T,read,carry,top,mb", [
    ("small", 5, 40, False, True, False, 8), ("small", 5, 40, True, True, True, 8), ("small", 4, 53, False, False, False, 8),
    ("q57low", 5, 33, True, False, True, 8), ("wide61", 4, 70, True, True, True, 13), ("wide", 5, 20, True, True, False, 0),
    ("wide61", 7, 17, False, True, True, 0), ("small", 3, 1040, False, False, False, 0)])
def test_segmented_prefix_sums(lib, orc, sets, monkeypatch, name, level, T, read, carry, top, mb):
    """A long chunk of one group: the tokens' prefix sums in segments, with the sums carried from one block of
    tokens to the next (mb MiB of intermediates, or 1024 tokens, a block), and with primes above 2^60."""
    ctx, P = sets(name)
    announce("segments %s level=%d T=%d read=%d carry=%d top=%d mb=%d" % (name, level, T, read, carry, top, mb))
    block = 1024
    if mb:
        monkeypatch.setenv("CKKS_BLOCK_MB", str(mb))
        limbs = 3 * (level + 1) + (2 * level if read else 0) + 2 * (level - 1) + 2 * (level - 2) + 3 * (level + 1)
        block = (mb << 17) // (limbs * P.N)
    assert min(T, block) >= 16 and (T < block or T - block >= 16)  # segments need 16 tokens
    st, ref_st = steps(lib, P, [2])
    rlk = key(P, 0, "rlk", top)
    d = chunk_case(P, level, T, 1, 1, read, carry, True, 40 + T, top)
    y, out = run_chunk(lib, ctx, P, d, level, T, 1, 1, rlk, st)
    ref = orc.linattn_chunk(P, level, d["q"], d["k"], d["v"], d["w"], d["r"], d["carry"], d["state"], rlk, *ref_st)
    same(y, ref[0], "y")
    same(out, ref[1], "state")


SETS.update({"full": (16, 6, 54, 2, 60, 3), "full57": (16, 4, 57, 2, 60, 2), "fullwide": (16, 4, 62, 2, 61, 2)})


@pytest.mark.parametrize("batch,radices", [(2, [3]), (3, [2]), (4, [3]), (5, [2]), (8, [2, 2])])
def test_full_ring_sums(lib, orc, sets, batch, radices):
    """N = 2^16: one group of 2 to 4 items a thread of the inner product, and several groups."""
    ctx, P = sets("full")
    announce("full ring sum batch=%d" % batch)
    st, (gal, keys) = steps(lib, P, radices)
    x = words(P, batch, "fs", 6, (batch, 2))
    out = empty_dev(x.shape)
    lib.ckks_rotate_sum(ctx, to_dev(x), out, batch, 5, st)
    same(out, np.stack([orc.rotate_sum(P, 5, c, gal, keys) for c in x]))


@pytest.mark.parametrize("name,level", [("full", 5), ("full57", 3), ("fullwide", 3)])
def test_full_ring_attention(lib, orc, sets, name, level):
    """N = 2^16: scores; a masked mix with its normaliser; a chunk with read weights, carry and state; a step:
    each size's own kernels, on lazy, 57-bit and 62-bit primes."""
    ctx, P = sets(name)
    announce("full ring %s" % name)
    st, ref_st = steps(lib, P, [2])
    rlk = key(P, 0, "rlk")
    d_rlk = to_dev(rlk)
    n = level + 1
    q, k = words(P, 1, "fq", n, (1, 2, 2)), words(P, 1, "fk", n, (1, 1, 2))
    s = empty_dev((1, 2, 1, 2, level, P.N))
    lib.ckks_attn_scores(ctx, to_dev(q), 2, to_dev(k), 1, 1, level, d_rlk, st, s)
    same(s, orc.attn_scores(P, level, q, k, rlk, *ref_st), "scores")
    a, v, m = words(P, 2, "fa", n, (1, 2, 2, 2)), words(P, 2, "fv", n, (1, 2, 2)), words(P, 2, "fm", n, (1, 2))
    num, den = empty_dev((1, 2, 2, level - 1, P.N)), empty_dev((1, 2, 2, level, P.N))
    lib.ckks_attn_mix(ctx, to_dev(a), 2, to_dev(v), 2, 1, to_dev(m), 1, level, d_rlk, st, num, den)
    ref = orc.attn_mix(P, level, a, v, m, rlk, *ref_st)
    same(num, ref[0], "num")
    same(den, ref[1], "den")
    d = chunk_case(P, level, 2, 1, 1, True, True, True, 3)
    y, out = run_chunk(lib, ctx, P, d, level, 2, 1, 1, rlk, st)
    ref = orc.linattn_chunk(P, level, d["q"], d["k"], d["v"], d["w"], d["r"], d["carry"], d["state"], rlk, *ref_st)
    same(y, ref[0], "chunk y")
    same(out, ref[1], "chunk state")
    q, k, v, s_in = (words(P, 4, "f" + t, n, (2, 2)) for t in "qkvs")
    dec = words(P, 4, "fd", n, (2,))
    y, out = empty_dev((2, 2, level - 1, P.N)), empty_dev((2, 2, level, P.N))
    lib.ckks_linattn_step(ctx, to_dev(q), to_dev(k), to_dev(v), 2, to_dev(dec), 2, to_dev(s_in), level, d_rlk, st, y, out)
    ref = orc.linattn_step(P, level, q, k, v, dec, s_in, rlk, *ref_st)
    same(y, ref[0], "step y")
    same(out, ref[1], "step state")


ONE_LANE = """
import sys
import numpy as np
import torch
import private_rns_ckks_amd as L

f = dict(np.load(sys.argv[1]))
dev = lambda k: torch.from_numpy(f[k].view(np.int64)).to("cuda")
log_n, dnum, lv = (int(f[k]) for k in ("log_n", "dnum", "lv"))
ctx = L.Context(log_n, f["q_mods"], f["p_mods"], dnum)
N = 1 << log_n
t = {k: dev(k) for k in ("a", "v", "m", "q", "k", "x", "w", "r", "carry", "s", "rlk", "evk")}
st = L.RotateSum([[int(f["g"])]], [[t["evk"]]])
new = lambda *shape: torch.full(shape, -1, dtype=torch.int64, device="cuda")
num, den = new(2, 2, lv - 1, N), new(2, 2, lv, N)
y, end = new(2, 2, lv - 2, N), new(1, 2, lv - 2, N)


def mix(groups, d):
    L.ckks_attn_mix(ctx, t["a"], 1, t["v"], 1, groups, t["m"], 1, lv, t["rlk"], st, num, d)


def chunk():
    L.ckks_linattn_chunk(ctx, t["q"], t["k"], t["x"], 2, 1, t["w"], t["r"], t["carry"], 1, t["s"], lv, t["rlk"], st, y, end)


for _ in range(2):
    mix(2, den)
    chunk()
torch.cuda.synchronize()
out = {"num": num, "den": den, "y": y, "end": end}
out = {k: o.cpu().numpy() for k, o in out.items()}
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
    mix(2, den)
    chunk()
for i in range(3):
    for o in (num, den, y, end):
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for k, o in (("num", num), ("den", den), ("y", y), ("end", end)):
        assert np.array_equal(o.cpu().numpy(), out[k]), (k, i)
fresh = L.Context(log_n, f["q_mods"], f["p_mods"], dnum)  # no call of it has created the internal streams
ctx = fresh
mix(2, None)
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
try:
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        mix(1, den)
    out["captured"] = np.array(1)
except L.CKKSError:
    out["captured"] = np.array(0)
np.savez(sys.argv[2], **out)
print("ONE_LANE ok", flush=True)
"""


@pytest.mark.parametrize("lanes", ["1", "2"])
def test_number_of_lanes(lib, orc, sets, tmp_path, lanes):
    """CKKS_LANES, read once a process: with 1 the calls that run steps side by side keep them on the caller's
    stream (a capture before any internal stream exists succeeds), with 2 on an internal stream (that capture is
    refused); the same words either way, captured ones too."""
    ctx, P = sets("small")
    announce("attention calls with CKKS_LANES=%s" % lanes)
    lv, n = 5, 6
    rlk, evk, g = key(P, 0, "rlk"), key(P, 0, "lane"), P.galois(3)
    c = {t: words(P, 1, "lane" + t, n, (2, 2)) for t in "avqkx"}
    p = {t: words(P, 1, "lane" + t, n, (2,)) for t in "wr"}
    m = words(P, 1, "lanem", n, (1,))
    carry, s_in = words(P, 1, "lanec", n - 2, (1,)), words(P, 1, "lanes", n - 2, (1, 2))
    np.savez(tmp_path / "in.npz", log_n=P.log_n, dnum=P.dnum, lv=lv, q_mods=np.array(P.q), p_mods=np.array(P.p), rlk=rlk,
             evk=evk, g=g, m=m, carry=carry, s=s_in, **c, **p)
    env = dict(os.environ, CKKS_LANES=lanes)
    r = subprocess.run([sys.executable, "-c", ONE_LANE, str(tmp_path / "in.npz"), str(tmp_path / "out.npz")], env=env,
                       cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "ONE_LANE ok" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
    got = {k: v.view(np.uint64) for k, v in np.load(tmp_path / "out.npz").items()}
    gal, keys = [[g]], [[evk]]
    rn, rd = orc.attn_mix(P, lv, c["a"][:, None, None], c["v"][:, None], m[:, None], rlk, gal, keys)
    ry, rs = orc.linattn_chunk(P, lv, c["q"][:, None], c["k"][:, None], c["x"][:, None], p["w"][:, None], p["r"][:, None],
                               carry, s_in, rlk, gal, keys)
    assert np.array_equal(got["num"], rn[:, 0]) and np.array_equal(got["den"], rd[:, 0])
    assert np.array_equal(got["y"], ry[:, 0]) and np.array_equal(got["end"], rs)
    assert int(got["captured"]) == (1 if lanes == "1" else 0)


def test_inputs_written_late_on_the_callers_stream(lib, orc, sets):
    """Inputs that a side stream writes only after long work of its own: the calls, enqueued before that, return
    without waiting for it and read the words it writes."""
    torch = torch_cuda()
    ctx, P = sets("mid")
    announce("late inputs")
    st, ref_st = steps(lib, P, [2])
    rlk = key(P, 0, "rlk")
    d_rlk = to_dev(rlk)
    lv, n = 5, 6
    names = ("a", "v", "q", "k", "x")
    host = {t: words(P, 2, "late" + t, n, (2, 2)) for t in names}
    pt = {t: words(P, 2, "late" + t, n, (2,)) for t in ("m", "w", "r")}
    carry, s_in = words(P, 2, "latec", n - 2, (1,)), words(P, 2, "lates", n - 2, (1, 2))
    src = {t: to_dev(x) for t, x in host.items()}
    d = {t: torch.zeros_like(x) for t, x in src.items()}
    p = {t: to_dev(x) for t, x in pt.items()}
    d_c, d_s = to_dev(carry), to_dev(s_in)
    outs = [empty_dev((2, 2, n, P.N)), empty_dev((1, 2, lv - 1, P.N)), empty_dev((1, 2, lv, P.N)),
            empty_dev((2, 2, lv - 2, P.N)), empty_dev((1, 2, lv - 2, P.N)), empty_dev((1, 2, 2, 2, lv, P.N)),
            empty_dev((2, 2, lv - 1, P.N)), empty_dev((2, 2, lv, P.N))]

    def calls():
        lib.ckks_rotate_sum(ctx, d["a"], outs[0], 2, lv, st)
        lib.ckks_attn_mix(ctx, d["a"], 1, d["v"], 2, 1, p["m"], 1, lv, d_rlk, st, outs[1], outs[2])
        lib.ckks_linattn_chunk(ctx, d["q"], d["k"], d["x"], 2, 1, p["w"], p["r"], d_c, 1, d_s, lv, d_rlk, st, outs[3],
                               outs[4])
        lib.ckks_attn_scores(ctx, d["q"], 2, d["k"], 2, 1, lv, d_rlk, st, outs[5])
        lib.ckks_linattn_step(ctx, d["q"], d["k"], d["x"], 2, None, 0, None, lv, d_rlk, st, outs[6], outs[7])

    side = torch.cuda.Stream()
    m = torch.ones((4096, 4096), device="cuda")
    with torch.cuda.stream(side):  # sizes the buffers, creates the internal streams, loads the kernels
        torch.mm(m, m)
        calls()
    torch.cuda.synchronize()
    busy = torch.cuda.Event()
    with torch.cuda.stream(side):
        for _ in range(200):  # some 200 ms
            acc = torch.mm(m, m)
        for t in names:
            d[t].copy_(src[t])
        busy.record()
        calls()
        waited = busy.query()
    side.synchronize()
    assert not waited, "a call waited for the stream's earlier work"
    assert float(acc[0, 0]) == 4096.0
    same(outs[0], np.stack([orc.rotate_sum(P, lv, c, *ref_st) for c in host["a"]]), "sum")
    rn, rd = orc.attn_mix(P, lv, host["a"][None, None], host["v"][None], pt["m"][None], rlk, *ref_st)
    same(outs[1], rn[0], "num")
    same(outs[2], rd[0], "den")
    ry, rs = orc.linattn_chunk(P, lv, host["q"][:, None], host["k"][:, None], host["x"][:, None], pt["w"][:, None],
                               pt["r"][:, None], carry, s_in, rlk, *ref_st)
    same(outs[3], ry[:, 0], "y")
    same(outs[4], rs, "state")
    same(outs[5], orc.attn_scores(P, lv, host["q"][None], host["k"][None], rlk, *ref_st), "scores")
    ry, rs = orc.linattn_step(P, lv, host["q"], host["k"], host["x"], None, None, rlk, *ref_st)
    same(outs[6], ry, "step y")
    same(outs[7], rs, "step state")


# Primes of several sizes in one context, as a chain of rescales has them: the
# conversions and rescales then cross sizes in both directions.
MIXED = {
    "mixed": (2, [60, 40, 54, 30, 57, 45], [60, 50, 36]),
    "mixedwide": (2, [62, 40, 61, 30, 54, 60], [61, 62, 50]),
}


def mixed_pair(lib, orc, log_n, dnum, q_bits, p_bits):
    taken = set()

    def pick(bits):
        m = next(v for v in lib.ckks_find_primes(log_n, bits, 9) if v not in taken)
        taken.add(m)
        return m

    q, p = [pick(b) for b in q_bits], [pick(b) for b in p_bits]
    return lib.Context(log_n, q, p, dnum), orc.Params(log_n, q, p, dnum)


@pytest.mark.parametrize("top", [False, True])
@pytest.mark.parametrize("log_n", [10, 13])
@pytest.mark.parametrize("name", list(MIXED))
def test_primes_of_several_sizes(lib, orc, name, log_n, top):
    ctx, P = mixed_pair(lib, orc, log_n, *MIXED[name])
    announce("mixed primes %s log_n=%d top=%d" % (name, log_n, top))
    st, ref_st = steps(lib, P, [3, 2], top=top)
    rlk = key(P, 0, "rlk", top)
    d_rlk = to_dev(rlk)
    for lv in (5, 4, 3):
        n = lv + 1
        a, v, m = words(P, lv, "ma", n, (2, 1, 2, 2), top), words(P, lv, "mv", n, (2, 2, 2), top), words(P, lv, "mm", n, (1, 2), top)
        num, den = empty_dev((2, 1, 2, lv - 1, P.N)), empty_dev((2, 1, 2, lv, P.N))
        lib.ckks_attn_mix(ctx, to_dev(a), 1, to_dev(v), 2, 2, to_dev(m), 1, lv, d_rlk, st, num, den)
        ref = orc.attn_mix(P, lv, a, v, m, rlk, *ref_st)
        same(num, ref[0], "num %d" % lv)
        same(den, ref[1], "den %d" % lv)
        d = chunk_case(P, lv, 2, 1, 1, True, True, True, lv, top)
        y, out = run_chunk(lib, ctx, P, d, lv, 2, 1, 1, rlk, st)
        ref = orc.linattn_chunk(P, lv, d["q"], d["k"], d["v"], d["w"], d["r"], d["carry"], d["state"], rlk, *ref_st)
        same(y, ref[0], "y %d" % lv)
        same(out, ref[1], "state %d" % lv)
        dec, s_in = words(P, lv, "mdec", n, (1,), top), words(P, lv, "ms", n, (1, 2), top)
        y, out = empty_dev((1, 2, lv - 1, P.N)), empty_dev((1, 2, lv, P.N))
        q, k, x = (to_dev(d[t][0]) for t in "qkv")
        lib.ckks_linattn_step(ctx, q, k, x, 1, to_dev(dec), 1, to_dev(s_in), lv, d_rlk, st, y, out)
        ref = orc.linattn_step(P, lv, d["q"][0], d["k"][0], d["v"][0], dec, s_in, rlk, *ref_st)
        same(y, ref[0], "step y %d" % lv)
        same(out, ref[1], "step state %d" % lv)
        s = empty_dev((2, 1, 2, 2, lv, P.N))
        lib.ckks_attn_scores(ctx, to_dev(a[:, :, 0]), 1, to_dev(v), 2, 2, lv, d_rlk, st, s)
        same(s, orc.attn_scores(P, lv, a[:, :, 0], v, rlk, *ref_st), "scores %d" % lv)
    ctx.close()


@pytest.mark.parametrize("shape,n_item", [((10, 20, 54, 5, 60, 4), 128), ((11, 20, 54, 5, 60, 4), 70),
                                          ((12, 24, 54, 8, 60, 3), 24), ((10, 20, 61, 5, 62, 4), 128)])
def test_many_items_on_small_rings(lib, orc, shape, n_item):
    """More limbs than the one-workgroup transforms take: small rings on the two-pass kernels, with one and two
    dropped limbs; the first, a middle and the last item against the oracle."""
    ctx, P = make_pair(lib, orc, *shape)
    lv = P.L - 1
    announce("%d items on a small ring %s" % (n_item, shape))
    assert n_item * (lv - 1) * P.N > 1 << 21
    st, ref_st = steps(lib, P, [2])
    rlk = key(P, 0, "rlk")
    d_rlk = to_dev(rlk)
    q, k = words(P, 1, "sq", lv + 1, (1, n_item, 2)), words(P, 1, "sk", lv + 1, (1, 1, 2))
    m = words(P, 1, "sm", lv + 1, (1, 1))
    d_q, d_k = to_dev(q), to_dev(k)
    pick = [0, n_item // 2, n_item - 1]
    s = empty_dev((1, n_item, 1, 2, lv, P.N))
    lib.ckks_attn_scores(ctx, d_q, n_item, d_k, 1, 1, lv, d_rlk, st, s)
    same(s[:, pick], orc.attn_scores(P, lv, q[:, pick], k, rlk, *ref_st), "scores")
    num, den = empty_dev((1, n_item, 2, lv - 1, P.N)), empty_dev((1, n_item, 2, lv, P.N))
    lib.ckks_attn_mix(ctx, d_q, n_item, d_k, 1, 1, to_dev(m), 1, lv, d_rlk, st, num, den)
    ref = orc.attn_mix(P, lv, q[:, pick, None], k, m, rlk, *ref_st)
    same(num[:, pick], ref[0], "num")
    same(den[:, pick], ref[1], "den")
    ctx.close()


@pytest.mark.parametrize("name,level,batch,features,radices", [
    ("small", 5, 2, 16, [4, 4]), ("c3", 12, 1, 64, [8, 8]), ("mid", 7, 5, 64, [8, 8]), ("mid14", 4, 1, 128, [2, 32, 2]),
    ("full", 5, 4, 64, [8, 8])])
def test_sums_of_the_outermost_index(lib, orc, sets, name, level, batch, features, radices):
    """The layout with the summed index outermost: rotations by multiples of n / F, whose automorphisms keep a word
    inside F adjacent ones."""
    ctx, P = sets(name)
    stride = P.N // 2 // features
    assert int(np.prod(radices)) == features
    announce("sum at stride n / %d on %s" % (features, name))
    st, (gal, keys) = steps(lib, P, radices, stride=stride)
    x = words(P, level, "outer", level + 1, (batch, 2))
    out = empty_dev(x.shape)
    lib.ckks_rotate_sum(ctx, to_dev(x), out, batch, level, st)
    same(out, np.stack([orc.rotate_sum(P, level, c, gal, keys) for c in x]))


def sized_calls(lib, P, st_two, st_one, d_rlk, lv, items):
    """The five calls on about `items` ciphertexts at `lv`: (name, function of a context, outputs)."""
    n, N = lv + 1, P.N
    w = lambda tag, limbs, *lead: to_dev(words(P, lv + 10 * items, "size" + tag, limbs, lead))
    x = {t: w(t, n, items, 2) for t in "qkva"}
    pt = {t: w("p" + t, n, items) for t in "mwrd"}
    made = []
    o = [empty_dev((items, 2, n, N))]
    made.append(("sum", lambda c, o=o: lib.ckks_rotate_sum(c, x["q"], o[0], items, lv, st_two), o))
    o = [empty_dev((items, 2, n, N))]
    made.append(("sum of one stage", lambda c, o=o: lib.ckks_rotate_sum(c, x["q"], o[0], items, lv, st_one), o))
    o = [empty_dev((items, 2, lv, N))]
    made.append(("scores", lambda c, o=o: lib.ckks_attn_scores(c, x["q"], items, x["k"], 1, 1, lv, d_rlk, st_two, o[0]), o))
    o = [empty_dev((items, 2, lv - 1, N)), empty_dev((items, 2, lv, N))]
    made.append(("mix", lambda c, o=o: lib.ckks_attn_mix(c, x["a"], 1, x["v"], 1, items, pt["m"], items, lv, d_rlk, st_two,
                                                         o[0], o[1]), o))
    o = [empty_dev((items, 2, lv - 1, N)), empty_dev((items, 2, lv, N))]
    s_in = w("s", n, items, 2)
    made.append(("step", lambda c, o=o: lib.ckks_linattn_step(c, x["q"], x["k"], x["v"], items, pt["d"], 1, s_in, lv, d_rlk,
                                                              st_two, o[0], o[1]), o))
    if lv >= 3:
        for G in (1, 2):
            T = items // G
            if not T:
                continue
            o = [empty_dev((T, G, 2, lv - 2, N)), empty_dev((G, 2, lv - 2, N))]
            carry, c_in = w("c", lv - 1, 1), w("cs", lv - 1, G, 2)
            made.append(("chunk of %d groups" % G, lambda c, o=o, T=T, G=G, carry=carry, c_in=c_in: lib.ckks_linattn_chunk(
                c, x["q"], x["k"], x["v"], T, G, pt["w"], pt["r"], carry, 1, c_in, lv, d_rlk, st_two, o[0], o[1]), o))
    return made


@pytest.mark.parametrize("mb", [1, 3])
def test_calls_no_larger_than_earlier_ones_can_be_captured(lib, orc, monkeypatch, mb):
    """After one call of each kind at the top level, the same kinds with fewer limbs or items need nothing new,
    also where blocks of a limited size hold more of the smaller items: each is captured and replayed."""
    torch = torch_cuda()
    monkeypatch.setenv("CKKS_BLOCK_MB", str(mb))
    ref_ctx, P = make_pair(lib, orc, *SETS["small"])
    announce("captures after larger calls, %d MiB" % mb)
    two, one = steps(lib, P, [2, 2])[0], steps(lib, P, [2])[0]
    d_rlk = to_dev(key(P, 0, "rlk"))
    kinds = [c[0] for c in sized_calls(lib, P, two, one, d_rlk, 5, 12)]
    failed = []
    for kind in kinds:
        ctx = make_pair(lib, orc, *SETS["small"])[0]
        first = "sum" if kind.startswith("sum") else kind
        dict((c[0], c[1]) for c in sized_calls(lib, P, two, one, d_rlk, 5, 12))[first](ctx)
        for lv in (5, 4, 3, 2):
            for items in (12, 9, 5, 2):
                call = next((c for c in sized_calls(lib, P, two, one, d_rlk, lv, items) if c[0] == kind), None)
                if call is None:
                    continue
                call[1](ref_ctx)
                torch.cuda.synchronize()
                ref = [o.clone() for o in call[2]]
                for o in call[2]:
                    o.zero_()
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                try:
                    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
                        call[1](ctx)
                except lib.CKKSError as e:
                    failed.append("%s level=%d items=%d: %s" % (kind, lv, items, e))
                    continue
                graph.replay()
                torch.cuda.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(call[2], ref)), (kind, lv, items)
                del graph
        ctx.close()
    assert not failed, "\n".join(failed)
    ref_ctx.close()


def test_block_limit_bounds_the_memory_of_a_call(lib, orc, sets, monkeypatch):
    """CKKS_BLOCK_MB limits the operand buffer and each of the (at most two) workspaces of a call: with 16 MiB, sums
    and mixes of 40 ciphertexts grow a new context by 3 x 16 MiB at most, where they would take over 200."""
    torch = torch_cuda()
    shape = SETS["mid"]
    ctx, P = sets("mid")
    announce("memory under a block limit")
    st, (gal, keys) = steps(lib, P, [2, 2])
    rlk = key(P, 0, "rlk")
    d_rlk = to_dev(rlk)
    n, B = 6, 40
    a, v = words(P, 1, "lima", n, (B, 2)), words(P, 1, "limv", n, (B, 2))
    m = words(P, 1, "limm", n, (1,))
    d_a, d_v, d_m = to_dev(a), to_dev(v), to_dev(m)
    o, num, den = empty_dev((B, 2, n, P.N)), empty_dev((B, 2, n - 2, P.N)), empty_dev((B, 2, n - 1, P.N))

    def calls(c):
        lib.ckks_rotate_sum(c, d_a, o, B, n - 1, st)
        lib.ckks_attn_mix(c, d_a, 1, d_v, 1, B, d_m, 1, n - 1, d_rlk, st, num, den)

    calls(ctx)  # loads the kernels, creates the device's streams
    fresh = make_pair(lib, orc, *shape)[0]
    lib.ckks_attn_mix(fresh, d_a, 1, d_v, 1, 1, d_m, 1, n - 1, d_rlk, st, num, den)
    torch.cuda.synchronize()
    for t in (o, num, den):
        t.zero_()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    monkeypatch.setenv("CKKS_BLOCK_MB", "16")
    calls(fresh)
    torch.cuda.synchronize()
    grown = before - torch.cuda.mem_get_info()[0]
    assert grown <= (3 * 16 + 6) << 20, grown  # allocations come in 2 MiB
    for b in (0, 1, B - 1):
        same(o[b], orc.rotate_sum(P, n - 1, a[b], gal, keys), "sum")
        ref = orc.attn_mix(P, n - 1, a[b, None, None, None], v[b, None, None], m[:, None], rlk, gal, keys)
        same(num[b], ref[0][0, 0], "num")
        same(den[b], ref[1][0, 0], "den")
    fresh.close()


@pytest.mark.parametrize("T,G,R,read,carry,state,radices", [
    (3, 5, 2, True, True, True, [2]), (4, 3, 3, False, True, False, []), (2, 6, 1, True, False, True, []),
    (7, 2, 2, False, False, False, [2, 2]), (1, 9, 4, True, True, False, [])])
def test_groups_and_tokens_in_small_blocks(lib, orc, sets, monkeypatch, T, G, R, read, carry, state, radices):
    """1 MiB of intermediates: a chunk's groups in several blocks with a carried state, with and without a sum."""
    monkeypatch.setenv("CKKS_BLOCK_MB", "1")
    ctx, P = sets("small")
    announce("small blocks T=%d G=%d R=%d read=%d carry=%d state=%d %s" % (T, G, R, read, carry, state, radices))
    st, ref_st = steps(lib, P, radices)
    rlk = key(P, 0, "rlk")
    d = chunk_case(P, 5, T, G, R, read, carry, state, 60 + T)
    y, out = run_chunk(lib, ctx, P, d, 5, T, G, R, rlk, st if radices else None)
    ref = orc.linattn_chunk(P, 5, d["q"], d["k"], d["v"], d["w"], d["r"], d["carry"], d["state"], rlk, *ref_st)
    same(y, ref[0], "y")
    same(out, ref[1], "state")


@pytest.mark.parametrize("M", [0, 2])
def test_unsummed_calls_in_small_blocks(lib, orc, sets, monkeypatch, M):
    """1 MiB of intermediates and no sum: blocks of scores, mixes (masked or not) and steps write their outputs in
    place."""
    monkeypatch.setenv("CKKS_BLOCK_MB", "1")
    ctx, P = sets("small")
    announce("unsummed small blocks M=%d" % M)
    rlk = key(P, 0, "rlk")
    d_rlk = to_dev(rlk)
    a, v, m = words(P, 8, "ua", 6, (3, 3, 2, 2)), words(P, 8, "uv", 6, (3, 2, 2)), words(P, 8, "um", 6, (max(M, 1), 2))
    low = 2 if M else 1
    num, den = empty_dev((3, 3, 2, 6 - low, P.N)), empty_dev((3, 3, 2, 7 - low, P.N))
    lib.ckks_attn_mix(ctx, to_dev(a), 3, to_dev(v), 2, 3, to_dev(m) if M else None, M, 5, d_rlk, None, num, den)
    ref = orc.attn_mix(P, 5, a, v, m if M else None, rlk, [], [])
    same(num, ref[0], "num")
    same(den, ref[1], "den")
    s = empty_dev((3, 3, 2, 2, 5, P.N))
    lib.ckks_attn_scores(ctx, to_dev(a[:, :, 0]), 3, to_dev(v), 2, 3, 5, d_rlk, None, s)
    same(s, orc.attn_scores(P, 5, a[:, :, 0], v, rlk, [], []), "scores")
    q, k, w = (words(P, 9, "u" + x, 6, (9, 2)) for x in "qkx")
    dec, s_in = (words(P, 9, "ud", 6, (M,)), words(P, 9, "us", 6, (9, 2))) if M else (None, words(P, 9, "us", 5, (9, 2)))
    y, out = empty_dev((9, 2, 4, P.N)), empty_dev((9, 2, 5, P.N))
    lib.ckks_linattn_step(ctx, to_dev(q), to_dev(k), to_dev(w), 9, dev(dec), M, to_dev(s_in), 5, d_rlk, None, y, out)
    ref = orc.linattn_step(P, 5, q, k, w, dec, s_in, rlk, [], [])
    same(y, ref[0], "y")
    same(out, ref[1], "state")
