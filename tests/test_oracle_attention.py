"""Pins for the oracle's attention on packed heads, and the binding's host
checks of the same calls (no GPU work).

Checked against what the mathematics fixes, on encrypted slots in float64:
  * a sum in stages leaves the sum over the axis in every slot of its cosets,
    whatever the radices, and one rotation is the hoisted rotation plus the
    input, word for word;
  * the chunked form of linear attention equals the recurrence
    S_t = gamma S_{t-1} + k_t v_t, y_t = q_t S_t summed over key features, with
    a decay for each head, a carried state and padded tokens;
  * the recurrent form equals the same recurrence, continuing a chunk's state;
  * cross attention with a polynomial weight p: sum_j m_j p(q k_j) v_j and
    sum_j m_j p(q k_j), a group whose mask leaves nothing giving zero.

Tolerance: 2^-20 of the largest value, the project's bound for decrypted
results.  Every encryption, key switch and rescale adds an error of about
sqrt(N h) sigma < 2^11 in units of one coefficient (N = 2^10, h = 64, sigma =
3.2), the sums here add fewer than 2^10 of them, a scale is at least 2^48 and
a decode sums N coefficients in quadrature (2^5): 2^(11 + 10 + 5 - 48) = 2^-22
of a unit value, and the outputs' largest value is at least 1."""
import ctypes
import os
import re

import numpy as np
import pytest

import ckks_synth as S
from helpers import encrypt_slots, galois_key, params, rel_err, relin_key, secret

TOL = 2.0 ** -20
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Scheme:
    """Keys and encryption for one small parameter set (50-bit primes near the scale)."""

    def __init__(self, orc, L=8, dnum=4):
        self.orc, self.P = orc, params(orc, 10, L, 50, -(-L // dnum), 60, dnum)
        self.n = self.P.N // 2
        self.s, self.s_ntt = secret(orc, self.P, 9, 64)
        self.rlk = relin_key(orc, self.P, self.s_ntt, 9)
        self.scale = 2.0 ** 50
        self.keys = {}

    def enc(self, z, level, tag, scale=None):
        return encrypt_slots(self.orc, self.P, self.s_ntt, np.asarray(z, dtype=np.complex128), scale or self.scale,
                             level, 9, tag)

    def pt(self, z, level, scale=None):
        return self.orc.encode(self.P, np.asarray(z, dtype=np.complex128), scale or self.scale, level)

    def dec(self, ct, scale):
        return self.orc.decrypt(self.P, ct.shape[-2] - 1, ct, self.s_ntt, scale).real

    def steps(self, stride, radices):
        """(galois, keys) of the sum over prod(radices) slots at `stride`."""
        gal, keys = [], []
        for r in radices:
            g = [self.P.galois(stride * k) for k in range(1, r)]
            gal.append(g)
            for v in g:
                if v not in self.keys:
                    self.keys[v] = galois_key(self.orc, self.P, self.s_ntt, v, 9, "g%d" % v)
            keys.append([self.keys[v] for v in g])
            stride *= r
        return gal, keys


@pytest.fixture(scope="module")
def sch(orc):
    return Scheme(orc)


@pytest.mark.parametrize("stride,radices", [(1, [8]), (64, [2, 4]), (16, [4, 8]), (8, [3]), (1, [4, 4, 4, 8])])
def test_rotate_sum_decrypts_to_the_sum(orc, sch, stride, radices):
    z = S.uniform_slots(S.stream(1, "sum"), sch.n, False)
    length = int(np.prod(radices))
    ct = sch.enc(z, 3, "sum")
    got = sch.dec(orc.rotate_sum(sch.P, 3, ct, *sch.steps(stride, radices)), sch.scale)
    ref = sum(np.roll(z.real, -stride * k) for k in range(length))
    assert rel_err(got, ref) < TOL


def test_rotate_sum_of_one_rotation_is_the_hoisted_rotation(orc, sch):
    ct = S.uniform_limbs(S.stream(2, "one"), sch.P.q[:6], sch.P.N, lead=(2,))
    gal, keys = sch.steps(5, [2])
    ref = orc.ct_add(sch.P, ct, orc.rotate_hoisted(sch.P, 5, ct, gal[0], keys[0])[0])
    assert np.array_equal(orc.rotate_sum(sch.P, 5, ct, gal, keys), ref)


def packed(n, F, heads):
    """Slot indices (feature, head, value feature) of the state layout."""
    return np.arange(n).reshape(F, heads, n // F // heads)


def linear_attention(n, F, heads, seed, T):
    """Random q, k, v and head decays on the state layout: slots with k and q
    replicated over value features and v over key features."""
    rng = S.stream(seed, "lin")
    d_v = n // F // heads
    q, k = (rng.uniform(-1, 1, (T, F, heads)) for _ in range(2))
    v = rng.uniform(-1, 1, (T, heads, d_v))
    gamma = 1.0 - 2.0 ** -(3.0 + np.arange(heads))
    rep = lambda x: np.broadcast_to(x[..., None], x.shape + (d_v,)).reshape(T, n)
    vv = np.broadcast_to(v[:, None], (T, F, heads, d_v)).reshape(T, n)
    g = np.broadcast_to(gamma[None, :, None], (F, heads, d_v)).reshape(n)
    return rep(q), rep(k), vv, g


def recurrence(q, k, v, g, F, state):
    ys = []
    for t in range(len(q)):
        state = g * state + k[t] * v[t]
        ys.append(np.tile((q[t] * state).reshape(F, -1).sum(0), F))
    return np.array(ys), state


def test_chunk_then_steps_equal_the_recurrence(orc, sch):
    n, F, heads, T, lv = sch.n, 8, 4, 3, 7
    q, k, v, g = linear_attention(n, F, heads, 3, T + 3)
    P, q_mod = sch.P, [float(x) for x in sch.P.q]
    gal, keys = sch.steps(n // F, [2, 4])
    start = S.uniform_slots(S.stream(3, "state"), n, False).real
    # scales: w (k x v), rescaled twice, is the state's; the carried state enters with it
    s_state = sch.scale ** 3 / q_mod[lv] / q_mod[lv - 1]
    ct = lambda x, tag: np.stack([sch.enc(a, lv, tag + str(i))[None] for i, a in enumerate(x)])
    w = np.stack([sch.pt(g ** -t, lv)[None] for t in range(T)])
    r = np.stack([sch.pt(g ** t, lv)[None] for t in range(T)])
    w[T - 1] = 0  # the last token is padding
    carry = np.stack([sch.pt(g ** (T - 1), lv - 2)])
    state = sch.enc(start, lv - 2, "st", s_state)[None]
    y, out = orc.linattn_chunk(P, lv, ct(q[:T], "q"), ct(k[:T], "k"), ct(v[:T], "v"), w, r, carry, state, sch.rlk, gal,
                               keys)
    # S_0 = start + k_0 v_0: the state that enters is the one before token 0, decayed once
    ref_y, ref_s = recurrence(q[: T - 1], k[: T - 1], v[: T - 1], g, F, start / g)
    s_y = sch.scale ** 2 / q_mod[lv] * s_state / q_mod[lv - 2]
    for t in range(T - 1):
        assert rel_err(sch.dec(y[t, 0], s_y), ref_y[t]) < TOL
    s_out = s_state * sch.scale / q_mod[lv - 2]
    assert rel_err(sch.dec(out[0], s_out), ref_s * g) < TOL  # carry = gamma^(T-1): one decay beyond S_(T-2)
    # recurrent steps from the chunk's state, at its level; the state's scale is met by the decay's
    ref, lv2, s_in, cur = ref_s * g, lv - 3, s_out, out
    for i in range(2):
        t = T + i
        dec = np.stack([sch.pt(g, lv2, sch.scale ** 2 / s_in)])
        one = lambda x, tag: sch.enc(x[t], lv2, tag + str(t))[None]
        yt, cur = orc.linattn_step(P, lv2, one(q, "q"), one(k, "k"), one(v, "v"), dec, cur, sch.rlk, gal, keys)
        s_in = sch.scale ** 2 / q_mod[lv2]
        ref_yt, ref = recurrence(q[t: t + 1], k[t: t + 1], v[t: t + 1], g, F, ref)
        assert rel_err(sch.dec(cur[0], s_in), ref) < TOL
        assert rel_err(sch.dec(yt[0], sch.scale * s_in / q_mod[lv2 - 1]), ref_yt[0]) < TOL
        lv2 -= 1


def test_step_without_decay_keeps_the_state_level(orc, sch):
    n, F = sch.n, 8
    q, k, v, _ = linear_attention(n, F, 4, 4, 3)
    gal, keys = sch.steps(n // F, [8])
    cur, ref, s = None, np.zeros(n), sch.scale ** 2 / float(sch.P.q[4])
    for t in range(3):
        one = lambda x, tag: sch.enc(x[t], 4, "n" + tag + str(t))[None]
        y, cur = orc.linattn_step(sch.P, 4, one(q, "q"), one(k, "k"), one(v, "v"), None, cur, sch.rlk, gal, keys)
        ref_y, ref = recurrence(q[t: t + 1], k[t: t + 1], v[t: t + 1], 1.0, F, ref)
        assert cur.shape[-2] == 4
        assert rel_err(sch.dec(cur[0], s), ref) < TOL
        assert rel_err(sch.dec(y[0], sch.scale * s / float(sch.P.q[3])), ref_y[0]) < TOL


def test_cross_attention_with_a_polynomial_weight(orc, sch):
    """Scores of 2 queries against 3 blocks of keys (the last one partly
    padded), weights p(s) = 1 + s + s^2 / 2, masked sums; the second group's
    mask leaves nothing."""
    n, F, lv, P = sch.n, 8, 7, sch.P
    toks = n // F
    rng = S.stream(5, "cross")
    q = np.repeat(rng.uniform(-0.5, 0.5, (2, 2, F, 1)), toks, axis=3).reshape(2, 2, n)
    k, v = (rng.uniform(-0.5, 0.5, (2, 3, F, toks)).reshape(2, 3, n) for _ in range(2))
    mask = np.zeros((2, 3, F, toks))
    mask[0] = 1.0
    mask[0, 2, :, toks // 3:] = 0.0
    mask = mask.reshape(2, 3, n)
    enc = lambda x, tag: np.array([[sch.enc(x[g, i], lv, "%s%d%d" % (tag, g, i)) for i in range(x.shape[1])]
                                   for g in range(2)])
    s = orc.attn_scores(P, lv, enc(q, "q"), enc(k, "k"), sch.rlk, *sch.steps(toks, [8]))
    s_score = sch.scale ** 2 / float(P.q[lv])
    ref_s = np.array([[[np.tile((q[g, i] * k[g, j]).reshape(F, toks).sum(0), F) for j in range(3)] for i in range(2)]
                      for g in range(2)])
    for g in range(2):
        for i in range(2):
            for j in range(3):
                assert rel_err(sch.dec(s[g, i, j], s_score), ref_s[g, i, j]) < TOL
    flat = s.reshape((12,) + s.shape[3:])
    p, s_p = orc.poly_eval_tree(P, lv - 1, flat, s_score, [1.0, 1.0, 0.5], sch.rlk)
    a = p.reshape((2, 2, 3) + p.shape[1:])
    la = a.shape[-2] - 1
    vs = np.array([[orc.encode(P, v[g, j].astype(complex), sch.scale, la) for j in range(3)] for g in range(2)])
    vct = np.stack([np.stack([np.stack([x, np.zeros_like(x)]) for x in row]) for row in vs])  # trivial encryptions
    m = np.array([[sch.pt(mask[g, j], la) for j in range(3)] for g in range(2)])
    num, den = orc.attn_mix(P, la, a, vct, m, sch.rlk, *sch.steps(1, [8, 8]))
    wgt = 1 + ref_s + ref_s ** 2 / 2
    s_den = s_p * sch.scale / float(P.q[la])
    s_num = s_p * sch.scale ** 2 / float(P.q[la]) / float(P.q[la - 1])
    first = np.arange(F) * toks  # token 0 of every feature holds the sum over the block's tokens
    for i in range(2):
        t = (mask[0] * wgt[0, i] * v[0]).sum(0).reshape(F, toks).sum(1)
        d = (mask[0] * wgt[0, i]).sum(0).reshape(F, toks).sum(1)
        assert rel_err(sch.dec(num[0, i], s_num)[first], t) < TOL
        assert rel_err(sch.dec(den[0, i], s_den)[first], d) < TOL
        assert np.abs(sch.dec(num[1, i], s_num)).max() < TOL
        assert np.abs(sch.dec(den[1, i], s_den)).max() < TOL


# ---------------------------------------------------------------- host checks

@pytest.fixture(scope="module")
def lib():
    import private_rns_ckks_amd as L

    return L


def test_null_context_is_refused(lib):
    f = lib.lib()
    assert f.ckks_rotate_sum(None, None, None, 1, 0, None, None) == lib.CKKS_EINVAL
    assert f.ckks_attn_scores(None, None, 1, None, 1, 1, 1, None, None, None, None) == lib.CKKS_EINVAL
    assert f.ckks_attn_mix(None, None, 1, None, 1, 1, None, 0, 1, None, None, None, None, None) == lib.CKKS_EINVAL
    assert f.ckks_linattn_chunk(None, None, None, None, 1, 1, None, None, None, 1, None, 3, None, None, None, None,
                                None) == lib.CKKS_EINVAL
    assert f.ckks_linattn_step(None, None, None, None, 1, None, 0, None, 2, None, None, None, None,
                               None) == lib.CKKS_EINVAL


class HostOnly:
    """The fields of a Context the binding's checks read."""
    handle, device, N, L, K, key_words = None, 0, 1024, 4, 1, 4 * 2 * 5 * 1024


def test_binding_refuses_before_the_library(lib):
    torch = pytest.importorskip("torch")
    ctx = HostOnly()
    x = torch.zeros((1, 2, 4, 1024), dtype=torch.int64)  # a host tensor
    with pytest.raises(lib.ArgumentError):
        lib.RotateSum([[5, 25]], [[x]])
    with pytest.raises(lib.ArgumentError):
        lib.RotateSum([[5], [25]], [[x]])
    st = lib.RotateSum([[5]], [[x]])
    assert st.radix == [2]
    with pytest.raises(lib.ArgumentError):
        st._c(ctx)
    for call in [lambda: lib.ckks_rotate_sum(ctx, x, x, 1, 3, st),
                 lambda: lib.ckks_attn_scores(ctx, x, 1, x, 1, 1, 3, x, st, x),
                 lambda: lib.ckks_attn_mix(ctx, x, 1, x, 1, 1, None, 0, 3, x, st, x),
                 lambda: lib.ckks_linattn_chunk(ctx, x, x, x, 1, 1, x, None, None, 1, None, 3, x, st, x, x),
                 lambda: lib.ckks_linattn_step(ctx, x, x, x, 1, None, 0, None, 3, x, st, x, x)]:
        with pytest.raises(lib.ArgumentError):
            call()


def test_sum_steps_structure_matches_the_header(lib):
    assert ctypes.sizeof(lib.ckks_sum_steps) == 32
    assert [f[0] for f in lib.ckks_sum_steps._fields_] == ["n_stage", "radix", "galois_elts", "d_evks"]


# ---------------------------------------------------------------- the documented weights

def header_weights():
    """Exponents of gamma that include/ckks.h gives the chunk's plaintexts, as functions of (u or t, n_tok)."""
    text = " ".join(line.strip(" *\n") for line in open(os.path.join(ROOT, "include", "ckks.h")))
    m = re.search(r"w_u = gamma\^(\S+), r_t = gamma\^(\S+) and carry = gamma\^(\w+)", text)
    assert m, "include/ckks.h no longer states the weights of a chunk"
    code = [compile(e, "ckks.h", "eval") for e in m.groups()]
    return [lambda i, n, c=c: eval(c, {"u": i, "t": i, "n_tok": n}) for c in code]


def test_a_prompt_by_the_documented_weights_continues_in_single_tokens(orc, sch):
    """A chunk with the header's w, r and carry, then steps with d_decay = gamma: one recurrence from the state
    before the prompt to the last token, the state that the chunk hands over among its values."""
    n, F, heads, T, lv = sch.n, 8, 4, 3, 7
    q, k, v, g = linear_attention(n, F, heads, 12, T + 2)
    q_mod = [float(x) for x in sch.P.q]
    gal, keys = sch.steps(n // F, [2, 4])
    start = S.uniform_slots(S.stream(12, "state"), n, False).real
    s_state = sch.scale ** 3 / q_mod[lv] / q_mod[lv - 1]
    ct = lambda x, tag: np.stack([sch.enc(a, lv, tag + str(i))[None] for i, a in enumerate(x)])
    e_w, e_r, e_carry = header_weights()
    w = np.stack([sch.pt(g ** float(e_w(t, T)), lv)[None] for t in range(T)])
    r = np.stack([sch.pt(g ** float(e_r(t, T)), lv)[None] for t in range(T)])
    carry = np.stack([sch.pt(g ** float(e_carry(None, T)), lv - 2)])
    y, cur = orc.linattn_chunk(sch.P, lv, ct(q[:T], "pq"), ct(k[:T], "pk"), ct(v[:T], "pv"), w, r, carry,
                               sch.enc(start, lv - 2, "pst", s_state)[None], sch.rlk, gal, keys)
    ref_y, ref = recurrence(q[:T], k[:T], v[:T], g, F, start)
    s_y = sch.scale ** 2 / q_mod[lv] * s_state / q_mod[lv - 2]
    for t in range(T):
        assert rel_err(sch.dec(y[t, 0], s_y), ref_y[t]) < TOL
    s_in, lv2 = s_state * sch.scale / q_mod[lv - 2], lv - 3
    assert rel_err(sch.dec(cur[0], s_in), ref) < TOL
    for t in range(T, T + 2):
        dec = np.stack([sch.pt(g, lv2, sch.scale ** 2 / s_in)])
        one = lambda x, tag: sch.enc(x[t], lv2, "p" + tag + str(t))[None]
        yt, cur = orc.linattn_step(sch.P, lv2, one(q, "q"), one(k, "k"), one(v, "v"), dec, cur, sch.rlk, gal, keys)
        s_in = sch.scale ** 2 / q_mod[lv2]
        ref_yt, ref = recurrence(q[t: t + 1], k[t: t + 1], v[t: t + 1], g, F, ref)
        assert rel_err(sch.dec(yt[0], sch.scale * s_in / q_mod[lv2 - 1]), ref_yt[0]) < TOL
        assert rel_err(sch.dec(cur[0], s_in), ref) < TOL
        lv2 -= 1


@pytest.mark.parametrize("strongest", [0.875, 0.5])
def test_a_chunk_loses_the_bits_of_its_decays(orc, sch, strongest):
    """The documented length of a chunk: with S_t up to gamma^-T larger than the state, the outputs of T tokens
    keep log2(gamma^-T) bits less than TOL gives for values of order 1: the errors that TOL bounds (2^-22 of a unit)
    meet a factor of at most gamma^-T (the sum's 2^10 terms, which TOL allows for, cover the state's size of a few
    units).  At 0.875 that is 1.5 bits, at 0.5 it is 8."""
    n, F, heads, T, lv = sch.n, 8, 4, 8, 5
    q, k, v, _ = linear_attention(n, F, heads, 13, T)
    gamma = np.linspace(strongest, 1.0, heads)
    g = np.broadcast_to(gamma[None, :, None], (F, heads, n // F // heads)).reshape(n)
    q_mod = [float(x) for x in sch.P.q]
    gal, keys = sch.steps(n // F, [8])
    ct = lambda x, tag: np.stack([sch.enc(a, lv, tag + str(i))[None] for i, a in enumerate(x)])
    e_w, e_r, e_carry = header_weights()
    w = np.stack([sch.pt(g ** float(e_w(t, T)), lv)[None] for t in range(T)])
    r = np.stack([sch.pt(g ** float(e_r(t, T)), lv)[None] for t in range(T)])
    carry = np.stack([sch.pt(g ** float(e_carry(None, T)), lv - 2)])
    y, cur = orc.linattn_chunk(sch.P, lv, ct(q, "lq"), ct(k, "lk"), ct(v, "lv"), w, r, carry, None, sch.rlk, gal, keys)
    s_state = sch.scale ** 3 / q_mod[lv] / q_mod[lv - 1]
    s_y = sch.scale ** 2 / q_mod[lv] * s_state / q_mod[lv - 2]
    ref_y, ref = recurrence(q, k, v, g, F, np.zeros(n))
    for t in range(T):
        assert rel_err(sch.dec(y[t, 0], s_y), ref_y[t]) < TOL * strongest ** -(t + 1)
    assert rel_err(sch.dec(cur[0], s_state * sch.scale / q_mod[lv - 2]), ref) < TOL * strongest ** -T
