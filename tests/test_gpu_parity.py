"""Bit-exact parity of the HIP library against the CPU oracle, through the C
interface, on seeded inputs: every output word must be equal.

Sizes span several NTT tiles and, where the shape allows, ragged counts
(odd batch sizes, partial last digits at lower levels, level 0, identity
Galois elements mixed into a batch)."""
import numpy as np
import pytest

import ckks_synth as S
from gpu_util import announce, config_pair, empty_dev, make_pair, misaligned_dev, to_dev, to_host, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    torch_cuda()
    import private_rns_ckks_amd as L

    return L


@pytest.fixture(scope="module")
def c1(lib, orc):
    return config_pair(lib, orc, "C1")


@pytest.fixture(scope="module")
def c3small(lib, orc):
    # C3 primes and digit structure at N = 2^12
    return config_pair(lib, orc, "C3", log_n=12)


# ---------------------------------------------------------------- NTT

@pytest.mark.parametrize("log_n", [10, 11, 12, 13, 14, 15, 16])
def test_ntt_parity_sizes(lib, orc, log_n):
    announce("ntt log_n=%d" % log_n)
    ctx, P = make_pair(lib, orc, log_n, 3, 54, 2, 60, 2)
    npoly, nl = 3, 5
    x = S.uniform_limbs(S.stream(log_n, "gpu/ntt"), P.mods, P.N, lead=(npoly,))
    d = to_dev(x)
    lib.ckks_ntt(ctx, d, npoly, 0, nl, 0)
    f = to_host(d)
    assert np.array_equal(f, orc.ntt_params(P, x))
    lib.ckks_ntt(ctx, d, npoly, 0, nl, 1)
    assert np.array_equal(to_host(d), x)
    # inverse on an independent input
    d2 = to_dev(x)
    lib.ckks_ntt(ctx, d2, npoly, 0, nl, 1)
    assert np.array_equal(to_host(d2), orc.ntt_params(P, x, inverse=True))


def test_ntt_limb_offset_and_edges(lib, orc, c3small):
    ctx, P = c3small
    announce("ntt limb_begin / edge values")
    x = S.uniform_limbs(S.stream(2, "gpu/ntt2"), P.mods[20:30], P.N, lead=(2,))
    x[0, 0, :7] = 0
    x[1, 3, :7] = np.uint64(P.mods[23] - 1)
    d = to_dev(x)
    lib.ckks_ntt(ctx, d, 2, 20, 10, 0)
    ref = orc.ntt(x, P.mods[20:30], P.psi[20:30], P.log_n)
    assert np.array_equal(to_host(d), ref)
    z = to_dev(np.zeros((1, 1, P.N), dtype=np.uint64))
    lib.ckks_ntt(ctx, z, 1, 31, 1, 0)
    assert not to_host(z).any()
    lib.ckks_ntt(ctx, d, 0, 0, 3, 0)  # empty batch is a no-op
    with pytest.raises(lib.CKKSError) as e:
        lib.ckks_ntt(ctx, d, 1, 30, 3, 0)
    assert e.value.code == lib.CKKS_ERANGE


def test_ntt_c2_full(lib, orc):
    """C2 at full size: 16 polynomials x 24 limbs x 2^16 words, forward then inverse."""
    announce("ntt C2 full")
    ctx, P = config_pair(lib, orc, "C2")
    x = S.uniform_limbs(S.stream(2, "C2/x"), P.q, P.N, lead=(16,))
    d = to_dev(x)
    lib.ckks_ntt(ctx, d, 16, 0, 24, 0)
    f = to_host(d)
    ref = orc.ntt_params(P, x)
    assert np.array_equal(f, ref)
    lib.ckks_ntt(ctx, d, 16, 0, 24, 1)
    assert np.array_equal(to_host(d), x)


# ---------------------------------------------------------------- automorphism

@pytest.mark.parametrize("domain", [0, 1])
def test_automorph_parity(lib, orc, c3small, domain):
    ctx, P = c3small
    level = 23
    announce("automorph domain=%d" % domain)
    x = S.uniform_limbs(S.stream(domain, "gpu/aut"), P.q, P.N, lead=(2,))
    dx = to_dev(x)
    out = empty_dev(x.shape)
    for g in [5, P.galois(7), 2 * P.N - 1, 1, P.galois(1234)]:
        lib.ckks_automorph(ctx, dx, out, 2, level, g, domain)
        got = to_host(out)
        if domain == 0:
            ref = orc.automorph_ntt(x, P.log_n, g)
        else:
            ref = orc.automorph_coeff(x, P.q, P.log_n, g)
        assert np.array_equal(got, ref), g
    with pytest.raises(lib.CKKSError) as e:
        lib.ckks_automorph(ctx, dx, out, 2, level, 4, domain)
    assert e.value.code == lib.CKKS_EINVAL


# ---------------------------------------------------------------- key switching

@pytest.mark.parametrize("level", [23, 16, 12, 7, 0])
def test_keyswitch_parity(lib, orc, c3small, level):
    ctx, P = c3small
    announce("keyswitch level=%d" % level)
    d = S.uniform_limbs(S.stream(level, "gpu/ks/d"), P.q[: level + 1], P.N)
    evk = S.uniform_limbs(S.stream(level, "gpu/ks/k"), P.mods, P.N, lead=(P.dnum, 2))
    out = empty_dev((2, level + 1, P.N))
    lib.ckks_keyswitch(ctx, to_dev(d), to_dev(evk), out, level)
    assert np.array_equal(to_host(out), orc.keyswitch(P, level, d, evk))


def test_keyswitch_parity_c1(lib, orc, c1):
    ctx, P = c1
    for level in (3, 1, 0):
        announce("keyswitch C1 level=%d" % level)
        d = S.uniform_limbs(S.stream(level, "gpu/ks1/d"), P.q[: level + 1], P.N)
        evk = S.uniform_limbs(S.stream(level, "gpu/ks1/k"), P.mods, P.N, lead=(P.dnum, 2))
        out = empty_dev((2, level + 1, P.N))
        lib.ckks_keyswitch(ctx, to_dev(d), to_dev(evk), out, level)
        assert np.array_equal(to_host(out), orc.keyswitch(P, level, d, evk))


# Parameter shapes beyond the workload recipes: every NTT pass geometry
# (log N 10..15), digits of one limb and of more than 8 limbs, more than 8
# special primes (the 16-source conversion path), a single digit, and
# ciphertext primes above 2^57 (no lazy butterflies on any limb).
KS_SHAPES = [
    # log_n, L, q_bits, K, p_bits, dnum, levels
    (10, 3, 40, 1, 50, 3, (2, 0)),
    (11, 10, 54, 10, 60, 1, (9, 4)),
    (12, 24, 54, 12, 60, 2, (23, 12, 11)),
    (13, 5, 54, 5, 60, 1, (4, 2)),
    (14, 8, 30, 4, 36, 2, (7, 3)),
    (15, 6, 59, 3, 60, 2, (5, 3, 0)),
]


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("shape", KS_SHAPES, ids=lambda s: "logn%d_L%d_q%d_K%d_dnum%d" % (s[0], s[1], s[2], s[3],
                                                                                          s[5]))
def test_rotate_shapes(lib, orc, shape, flags):
    """Rotations (the automorphism gathered inside the key switch, with and
    without accumulation) over every key-switch shape: log N 10..15, one-limb
    and 10-12-limb digits, 10-12 special primes, 59-bit ciphertext primes."""
    log_n, L, q_bits, K, p_bits, dnum, levels = shape
    ctx, P = make_pair(lib, orc, log_n, L, q_bits, K, p_bits, dnum)
    for level in levels:
        announce("rotate shape %s level=%d flags=%d" % (shape[:6], level, flags))
        ks = [1, 3, P.N // 2 - 5]
        cts = S.uniform_limbs(S.stream(level, "gpu/rots/ct"), P.q[: level + 1], P.N, lead=(len(ks), 2))
        gs = [P.galois(k) for k in ks]
        keys = [S.uniform_limbs(S.stream(b, "gpu/rots/k"), P.mods, P.N, lead=(P.dnum, 2)) for b in range(len(ks))]
        out = empty_dev(cts.shape)
        lib.ckks_rotate(ctx, to_dev(cts), out, len(ks), level, gs, [to_dev(k) for k in keys], flags)
        ref = orc.rotate_batch(P, level, cts, gs, keys, orc.ROT_ACCUMULATE if flags else 0)
        assert np.array_equal(to_host(out), ref), level
    ctx.close()


@pytest.mark.parametrize("shape", KS_SHAPES, ids=lambda s: "logn%d_L%d_K%d_dnum%d" % (s[0], s[1], s[3], s[5]))
def test_keyswitch_shapes(lib, orc, shape):
    log_n, L, q_bits, K, p_bits, dnum, levels = shape
    ctx, P = make_pair(lib, orc, log_n, L, q_bits, K, p_bits, dnum)
    for level in levels:
        announce("keyswitch shape %s level=%d" % (shape[:6], level))
        d = S.uniform_limbs(S.stream(level, "gpu/kss/d"), P.q[: level + 1], P.N)
        evk = S.uniform_limbs(S.stream(level, "gpu/kss/k"), P.mods, P.N, lead=(P.dnum, 2))
        out = empty_dev((2, level + 1, P.N))
        lib.ckks_keyswitch(ctx, to_dev(d), to_dev(evk), out, level)
        assert np.array_equal(to_host(out), orc.keyswitch(P, level, d, evk)), level
    ctx.close()


# ---------------------------------------------------------------- rotation

def test_rotate_c1_encrypted(lib, orc, c1):
    """C1: real encryption, rotate by 1 and by 7; words equal the oracle's and decrypt to the shift."""
    from helpers import encrypt_slots, galois_key, rel_err, secret

    ctx, P = c1
    c = S.CONFIGS["C1"]
    announce("rotate C1")
    s, s_ntt = secret(orc, P, 1, c["h"])
    z = S.uniform_slots(S.stream(1, "msg"), P.N // 2, complex_values=True)
    level = P.L - 1
    ct = encrypt_slots(orc, P, s_ntt, z, c["scale"], level, 1, "ct")
    for k in c["rotations"]:
        g = P.galois(k)
        evk = galois_key(orc, P, s_ntt, g, 1, "gk%d" % k)
        out = empty_dev(ct.shape)
        lib.ckks_rotate(ctx, to_dev(ct), out, 1, level, [g], [to_dev(evk)])
        got = to_host(out)
        assert np.array_equal(got, orc.rotate(P, level, ct, g, evk))
        assert rel_err(orc.decrypt(P, level, got, s_ntt, c["scale"]), np.roll(z, -k)) < 2 ** -12


@pytest.mark.parametrize("flags", [0, 1])
def test_rotate_batch_mixed(lib, orc, c3small, flags):
    ctx, P = c3small
    level = 22
    B = 7
    announce("rotate batch mixed flags=%d" % flags)
    cts = S.uniform_limbs(S.stream(flags, "gpu/rot/ct"), P.q[: level + 1], P.N, lead=(B, 2))
    gs = [P.galois(k) for k in (1, 3, 0, 100, 2047, 5, 0)]
    keys_h = [S.uniform_limbs(S.stream(b, "gpu/rot/k"), P.mods, P.N, lead=(P.dnum, 2)) for b in range(B)]
    keys = [to_dev(k) for k in keys_h]
    out = empty_dev(cts.shape)
    lib.ckks_rotate(ctx, to_dev(cts), out, B, level, gs, keys, flags)
    got = to_host(out)
    ref = orc.rotate_batch(P, level, cts, gs, keys_h, flags)
    assert np.array_equal(got, ref)


def test_rotate_batch_chunks(lib, orc, c3small):
    """Runs of 5, 1 and 6 key-switched items between identity items: chunks of
    4, 1, 1, 4 and 2 items spread over the internal streams."""
    ctx, P = c3small
    level = 20
    ks = [1, 2, 3, 4, 5, 0, 6, 0, 7, 8, 9, 10, 11, 12]
    B = len(ks)
    announce("rotate batch of %d in chunks" % B)
    cts = S.uniform_limbs(S.stream(5, "gpu/rotc/ct"), P.q[: level + 1], P.N, lead=(B, 2))
    gs = [P.galois(k) for k in ks]
    keys_h = [S.uniform_limbs(S.stream(b, "gpu/rotc/k"), P.mods, P.N, lead=(P.dnum, 2)) for b in range(B)]
    out = empty_dev(cts.shape)
    lib.ckks_rotate(ctx, to_dev(cts), out, B, level, gs, [to_dev(k) for k in keys_h], lib.CKKS_ROT_ACCUMULATE)
    got = to_host(out)
    ref = orc.rotate_batch(P, level, cts, gs, keys_h, orc.ROT_ACCUMULATE)
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("level", [23, 12])
def test_rotate_hoisted_parity(lib, orc, c3small, level):
    """Hoisted rotations of 3 inputs by 6 elements (one the identity), in
    chunks across the internal streams, against the oracle's hoisted rotation."""
    ctx, P = c3small
    ks = [1, 3, 0, 100, 2047, 5]
    n_in, R = 3, len(ks)
    announce("hoisted rotations level=%d" % level)
    cts = S.uniform_limbs(S.stream(level, "gpu/hoist/ct"), P.q[: level + 1], P.N, lead=(n_in, 2))
    gs = [P.galois(k) for k in ks]
    keys_h = [S.uniform_limbs(S.stream(r, "gpu/hoist/k"), P.mods, P.N, lead=(P.dnum, 2)) for r in range(R)]
    out = empty_dev((n_in, R) + cts.shape[1:])
    lib.ckks_rotate_hoisted(ctx, to_dev(cts), n_in, level, gs, [to_dev(k) for k in keys_h], out)
    got = to_host(out)
    for c in range(n_in):
        assert np.array_equal(got[c], orc.rotate_hoisted(P, level, cts[c], gs, keys_h)), c


def test_rotate_hoisted_c1_encrypted(lib, orc, c1):
    """C1: real encryption, four hoisted rotations; words equal the oracle's and decrypt to the shifts."""
    from helpers import encrypt_slots, galois_key, rel_err, secret

    ctx, P = c1
    c = S.CONFIGS["C1"]
    level = P.L - 1
    s, s_ntt = secret(orc, P, 4, c["h"])
    z = S.uniform_slots(S.stream(4, "gpu/hc1/msg"), P.N // 2, complex_values=True)
    ct = encrypt_slots(orc, P, s_ntt, z, c["scale"], level, 4, "gpu/hc1/ct")
    ks = [1, 2, 7, 100]
    gs = [P.galois(k) for k in ks]
    keys_h = [galois_key(orc, P, s_ntt, g, 4, "gpu/hc1/k%d" % g) for g in gs]
    out = empty_dev((1, len(ks)) + ct.shape)
    lib.ckks_rotate_hoisted(ctx, to_dev(ct[None]), 1, level, gs, [to_dev(k) for k in keys_h], out)
    got = to_host(out)[0]
    ref = orc.rotate_hoisted(P, level, ct, gs, keys_h)
    assert np.array_equal(got, ref)
    for r, k in enumerate(ks):
        assert rel_err(orc.decrypt(P, level, got[r], s_ntt, c["scale"]), np.roll(z, -k)) < 2 ** -12, k


def test_rotate_errors(lib, orc, c3small):
    ctx, P = c3small
    x = empty_dev((1, 2, 24, P.N))
    y = empty_dev((1, 2, 24, P.N))
    k = empty_dev((3, 2, 32, P.N))
    for args, code in [((1, 24, [5], [k]), lib.CKKS_ERANGE), ((1, 23, [6], [k]), lib.CKKS_EINVAL),
                       ((1, 23, [2 * P.N + 1], [k]), lib.CKKS_EINVAL), ((1, -1, [5], [k]), lib.CKKS_ERANGE)]:
        with pytest.raises(lib.CKKSError) as e:
            lib.ckks_rotate(ctx, x, y, *args)
        assert e.value.code == code
    # buffers must be 16-byte aligned; rejected on the host before any launch
    for a_in, keys in [(x, [misaligned_dev(k.shape)]), (misaligned_dev(x.shape), [k])]:
        with pytest.raises(lib.CKKSError) as e:
            lib.ckks_rotate(ctx, a_in, y, 1, 23, [5], keys)
        assert e.value.code == lib.CKKS_EINVAL
    # an output overlapping the input or a key races with the kernels that read them
    z = empty_dev((3, 2, 24, P.N))
    shifted = z.view(-1)[P.N: P.N + 2 * 24 * P.N].view(1, 2, 24, P.N)  # overlaps z[0] by all but one limb
    for a_in, out, keys in [(x, x, [k]), (z[:1], shifted, [k]),
                            (x, k.view(-1)[: 2 * 24 * P.N].view(1, 2, 24, P.N), [k])]:
        with pytest.raises(lib.CKKSError) as e:
            lib.ckks_rotate(ctx, a_in, out, 1, 23, [5], keys)
        assert e.value.code == lib.CKKS_EINVAL


def test_binding_argument_checks(lib, orc, c3small):
    """The binding rejects what the library cannot see (list lengths, tensor
    sizes, devices, a missing key) on the host, before any call."""
    torch = torch_cuda()
    ctx, P = c3small
    x = empty_dev((2, 2, 24, P.N))
    y = empty_dev((2, 2, 24, P.N))
    k = empty_dev((3, 2, 32, P.N))
    bad = [
        lambda: lib.ckks_rotate(ctx, x, y, 2, 23, [5], [k, k]),             # one Galois element for two items
        lambda: lib.ckks_rotate(ctx, x, y, 2, 23, [5, 25], [k]),            # one key for two items
        lambda: lib.ckks_rotate(ctx, x, y, 3, 23, [5, 25, 5], [k, k, k]),   # batch larger than the tensors
        lambda: lib.ckks_rotate(ctx, x, y, 1, 23, [5], [k.view(-1)[: P.N]]),  # short key
        lambda: lib.ckks_rotate(ctx, x, y, 1, 23, [5], [None]),             # missing key
        lambda: lib.ckks_rotate(ctx, x.cpu(), y, 1, 23, [5], [k]),          # host tensor
        lambda: lib.ckks_rotate(ctx, x, y[:, :, :, :8], 1, 23, [5], [k]),   # non-contiguous view
        lambda: lib.ckks_keyswitch(ctx, x, k, y.view(-1)[: P.N], 23),       # short output
        lambda: lib.ckks_rescale(ctx, x, y, 3, 23),
        lambda: lib.ckks_mul_relin_rescale(ctx, x, x.view(-1)[:5], k, y, 1, 23),
        lambda: lib.ckks_ntt(ctx, x, 5, 0, 24, 0),                          # 5 x 24 limbs in a 4 x 24 tensor
        lambda: lib.ckks_rotate_hoisted(ctx, x, 1, 23, [5, 25], [k], y),
        lambda: lib.ckks_ptmatvec(ctx, x, 1, empty_dev((1, 1, 2, 2, 24, P.N)), 1, 2, 2, [5], [], [25], [k], y, 23),
        lambda: lib.ckks_ctmatvec(ctx, x, 1, empty_dev((1, 1, 2, 2, 24, P.N)), 1, 2, 2, k, [5], [k], [25], [k], y,
                                  23),  # plaintext-sized diagonals for ciphertext diagonals
    ]
    for i, f in enumerate(bad):
        with pytest.raises(lib.ArgumentError):
            f()
    torch.cuda.synchronize()
    # a missing key is allowed for the identity element (a copy)
    lib.ckks_rotate(ctx, x, y, 1, 23, [1], [None])


def test_overlap_rejected(lib, orc, c3small):
    """Every call with an output rejects outputs that overlap its inputs or keys (CKKS_EINVAL)."""
    ctx, P = c3small
    x = empty_dev((2, 2, 24, P.N))
    k = empty_dev((3, 2, 32, P.N))
    ks = [k.view(-1)[: 2 * 24 * P.N * 2].view(2, 2, 24, P.N)]
    calls = [
        lambda: lib.ckks_automorph(ctx, x, x, 2, 23, 5, 0),
        lambda: lib.ckks_keyswitch(ctx, x[0, 1], k, x[0], 23),
        lambda: lib.ckks_keyswitch(ctx, x[0, 1], k, ks[0][0], 23),
        lambda: lib.ckks_rotate_hoisted(ctx, x[:1], 1, 23, [5, 25], [k, k], x),
        lambda: lib.ckks_rescale(ctx, x, x, 2, 23),
        lambda: lib.ckks_mul_relin_rescale(ctx, x, x, k, x, 1, 23, lib.CKKS_NO_RESCALE),
        lambda: lib.ckks_mul_relin_rescale(ctx, x[:1], x[1:], k, ks[0][:1], 1, 23, lib.CKKS_NO_RESCALE),
        lambda: lib.ckks_poly_eval(ctx, x, 1, 23, 2.0 ** 54, [0.5, 1.0], k, x),
        lambda: lib.ckks_poly_eval_tree(ctx, x, 1, 23, 2.0 ** 54, [0.5, 1.0, 0.25], k, x),
        lambda: lib.ckks_ptmatvec(ctx, x[:1], 1, empty_dev((1, 1, 2, 2, 24, P.N)), 1, 2, 2, [5], [k], [25], [k],
                                  x[:1], 23, lib.CKKS_NO_RESCALE),
        lambda: lib.ckks_ctmatvec(ctx, x[:1], 1, empty_dev((1, 1, 2, 2, 2, 24, P.N)), 1, 2, 2, k, [5], [k], [25],
                                  [k], ks[0][:1], 23, lib.CKKS_NO_RESCALE),
    ]
    for i, f in enumerate(calls):
        with pytest.raises(lib.CKKSError) as e:
            f()
        assert e.value.code == lib.CKKS_EINVAL, i
        assert "overlap" in lib.ckks_last_error(), i


def test_keyswitch_debug_dump_localises_stages(lib, orc, c3small, tmp_path, monkeypatch):
    """CKKS_DEBUG_DUMP writes the key switch's intermediates; each is checked
    against its definition, computed here from the oracle's transforms and
    conversions, so a mismatch names its stage: the ModUp inputs
    y_i = x_i [qhat_i^-1], the ModUp conversion, the special accumulators'
    y_k = iNTT(sum_j NTT(modup_j) evk_j) [phat_k^-1] and the ModDown
    conversion sum_k y_k [1/p_k]_{q_i} - #{y_k > (p_k-1)/2}."""
    import glob
    import os

    ctx, P = c3small
    level = 13  # two digits, the second partial
    nq, N = level + 1, P.N
    announce("keyswitch debug dump level=%d" % level)
    d = S.uniform_limbs(S.stream(3, "gpu/dump/d"), P.q[:nq], N)
    evk = S.uniform_limbs(S.stream(3, "gpu/dump/k"), P.mods, N, lead=(P.dnum, 2))
    monkeypatch.setenv("CKKS_DEBUG_DUMP", str(tmp_path))
    out = empty_dev((2, nq, N))
    lib.ckks_keyswitch(ctx, to_dev(d), to_dev(evk), out, level)
    monkeypatch.delenv("CKKS_DEBUG_DUMP")
    assert np.array_equal(to_host(out), orc.keyswitch(P, level, d, evk))
    seq = max(os.path.basename(f)[2:8] for f in glob.glob(str(tmp_path / "ks*_modup_in_item0.u64")))

    def dump(stage, shape):
        return np.fromfile(str(tmp_path / ("ks%s_%s_item0.u64" % (seq, stage))), dtype=np.uint64).reshape(shape)

    x = orc.ntt_params(P, d, inverse=True)  # coefficient form
    beta, alpha, K = P.beta(level), P.alpha, P.K
    next_ = nq + K
    ext = P.ext_mods(level)
    # modup_in
    y = dump("modup_in", (nq, N))
    for j in range(beta):
        lo, hi = j * alpha, min((j + 1) * alpha, nq)
        for i in range(lo, hi):
            qi = P.q[i]
            qhat = 1
            for t in range(lo, hi):
                if t != i:
                    qhat *= P.q[t]
            c = pow(qhat % qi, -1, qi)
            assert [int(v) for v in y[i]] == [int(v) * c % qi for v in x[i]], ("modup_in", i)
    # modup_out
    e = dump("modup_out", (beta, next_, N))
    mu = [orc.modup(P, level, j, x) for j in range(beta)]
    for j in range(beta):
        lo, hi = j * alpha, min((j + 1) * alpha, nq)
        for t in range(next_):
            if lo <= t < hi:
                continue
            m = ext[t]
            assert np.array_equal(e[j, t] % np.uint64(m), mu[j][t]), ("modup_out", j, t)
    # moddown_in
    a = dump("moddown_in", (2, K, N))
    psi_p = P.psi[P.L:]
    Pprod = 1
    for pk in P.p:
        Pprod *= pk
    ys = np.zeros((2, K, N), dtype=object)
    for k, pk in enumerate(P.p):
        acc = [np.zeros(N, dtype=object), np.zeros(N, dtype=object)]
        for j in range(beta):
            f = orc.ntt(mu[j][nq + k][None], [pk], [psi_p[k]], P.log_n)[0].astype(object)
            for comp in range(2):
                acc[comp] = (acc[comp] + f * evk[j, comp, P.L + k].astype(object)) % pk
        phinv = pow((Pprod // pk) % pk, -1, pk)
        for comp in range(2):
            coeff = orc.ntt(np.array(acc[comp], dtype=np.uint64)[None], [pk], [psi_p[k]], P.log_n, inverse=True)[0]
            ys[comp, k] = coeff.astype(object) * phinv % pk
            assert [int(v) for v in a[comp, k]] == list(ys[comp, k]), ("moddown_in", comp, k)
    # moddown_out
    w = dump("moddown_out", (2, nq, N))
    for comp in range(2):
        neg = sum((ys[comp, k] > (pk - 1) // 2).astype(object) for k, pk in enumerate(P.p))
        for i in range(nq):
            qi = P.q[i]
            ref = sum(ys[comp, k] * pow(pk % qi, -1, qi) for k, pk in enumerate(P.p)) - neg
            assert [int(v) % qi for v in w[comp, i]] == [int(v) % qi for v in ref], ("moddown_out", comp, i)


# ---------------------------------------------------------------- polynomial evaluation

@pytest.mark.parametrize("coeffs,level", [
    ([1.0, 1.0, 0.5, 1 / 6, 1 / 24, 1 / 120, 1 / 720, 1 / 5040], 23),
    ([-1.75, 0.3, 1.9, -0.6], 9),
    ([0.25, -1.5], 4),
    ([0.1, 0.0, 2.5], 3),
], ids=["exp7_l23", "cubic_l9", "affine_l4", "quad_l3"])
def test_poly_eval_parity(lib, orc, c3small, coeffs, level):
    """Horner evaluation on 3 ciphertexts; item 0 a real encryption at scale
    2^54 that decrypts to the polynomial of its slots."""
    from helpers import encrypt_slots, relin_key, secret

    ctx, P = c3small
    d = len(coeffs) - 1
    announce("poly_eval degree=%d level=%d" % (d, level))
    s, s_ntt = secret(orc, P, 11, 192)
    rlk = relin_key(orc, P, s_ntt, 11, tag="gpu/pe/rlk")
    scale = 2.0 ** 54
    cts = S.uniform_limbs(S.stream(level, "gpu/pe/ct"), P.q[: level + 1], P.N, lead=(3, 2))
    z = S.uniform_slots(S.stream(level, "gpu/pe/z"), P.N // 2, complex_values=False)
    cts[0] = encrypt_slots(orc, P, s_ntt, z, scale, level, 11, "gpu/pe/enc")
    out = empty_dev((3, 2, level - d + 1, P.N))
    s_out = lib.ckks_poly_eval(ctx, to_dev(cts), 3, level, scale, coeffs, to_dev(rlk), out)
    got = to_host(out)
    ref, ref_scale = orc.poly_eval(P, level, cts, scale, coeffs, rlk)
    assert s_out == ref_scale
    assert np.array_equal(got, ref)
    dec = orc.decrypt(P, level - d, got[0], s_ntt, s_out).real
    assert np.max(np.abs(dec - sum(c * z ** k for k, c in enumerate(coeffs)))) < 2 ** -30


def test_poly_eval_errors(lib, orc, c3small):
    ctx, P = c3small
    x = empty_dev((1, 2, 3, P.N))
    k = empty_dev((3, 2, 32, P.N))
    y = empty_dev((1, 2, 3, P.N))
    for level, coeffs, code in [(2, [1.0] * 4, lib.CKKS_ERANGE), (2, [1.0], lib.CKKS_ERANGE),
                                (2, [0.0, 2.0 ** 40], lib.CKKS_EINVAL)]:
        with pytest.raises(lib.CKKSError) as e:
            lib.ckks_poly_eval(ctx, x, 1, level, 2.0 ** 54, coeffs, k, y)
        assert e.value.code == code


def _cheb_fit(f, degree, lo, hi):
    from numpy.polynomial import chebyshev as C, polynomial as Pm
    p = C.Chebyshev.interpolate(f, degree, domain=[lo, hi]).convert(kind=Pm.Polynomial, domain=[-1, 1],
                                                                   window=[-1, 1])
    return [float(v) for v in p.coef]


def _gelu_fit():
    import math

    c = _cheb_fit(lambda u: 2.0 * u * (1.0 + np.vectorize(math.erf)(4.0 * u / math.sqrt(2.0))), 15, -1.0, 1.0)
    for k in range(3, 16, 2):  # GELU(x) - x/2 is even
        c[k] = 0.0
    return c


TREE_CASES = [
    ("exp7_l23", [1.0, 1.0, 0.5, 1 / 6, 1 / 24, 1 / 120, 1 / 720, 1 / 5040], 23, 3, None),
    ("exp11_m4_0_l23", None, 23, 3, "exp"),                   # x in [-4, 0] directly: powers up to 4^8
    ("exp11_u_l23", None, 23, 3, "exp_u"),                    # u = x/4 in [-1, 0], fit of exp(4u)
    ("gelu15_l23", None, 23, 3, "gelu"),
    ("deg16_l8", [0.1 * (-1) ** k / (k + 1) for k in range(17)], 8, 3, None),
    ("cubic_l5_b18", [-1.75, 0.3, 1.9, -0.6], 5, 18, None),   # two chunks of items
    ("affine_l1", [0.25, -1.5], 1, 3, None),
    ("quad_no_x_l2", [0.1, 0.0, 2.5], 2, 3, None),            # output at level 0
    ("quad_no_x_l4", [0.1, 0.0, 2.5], 4, 3, None),
    ("const_only_l1", [0.3, 0.0], 1, 3, None),                # every term zero: a trivial ciphertext
    ("x_only_l3", [0.0, 1.0], 3, 3, None),
    ("x8_l6", [0.3, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, -0.7], 6, 3, None),   # one-coefficient high part
    ("deg31_l12", [0.2 * (k % 3 - 1) for k in range(32)], 12, 2, None),      # zero runs, depth 5
]


@pytest.mark.parametrize("name,coeffs,level,B,fn", TREE_CASES, ids=[c[0] for c in TREE_CASES])
def test_poly_eval_tree_parity(lib, orc, c3small, name, coeffs, level, B, fn):
    """Depth-efficient evaluation on B ciphertexts, word for word against the
    oracle; item 0 a real encryption at scale 2^54 that decrypts to the
    polynomial (exp: inputs in [-4, 0]; GELU: u = x/4 in [-1, 1])."""
    from helpers import encrypt_slots, relin_key, secret

    ctx, P = c3small
    if fn == "exp":
        coeffs = _cheb_fit(np.exp, 11, -4.0, 0.0)
    elif fn == "exp_u":
        coeffs = _cheb_fit(lambda u: np.exp(4.0 * u), 11, -1.0, 0.0)
    elif fn == "gelu":
        coeffs = _gelu_fit()
    d = len(coeffs) - 1
    depth = lib.tree_depth(d)
    announce("poly_eval_tree %s degree=%d level=%d batch=%d" % (name, d, level, B))
    s, s_ntt = secret(orc, P, 12, 192)
    rlk = relin_key(orc, P, s_ntt, 12, tag="gpu/pt/rlk")
    scale = 2.0 ** 54
    cts = S.uniform_limbs(S.stream(level, "gpu/pt/ct"), P.q[: level + 1], P.N, lead=(B, 2))
    rng = S.stream(level, "gpu/pt/z")
    if fn == "exp":
        z = -4.0 * rng.random(P.N // 2)
    elif fn == "exp_u":
        z = -rng.random(P.N // 2)
    else:
        z = S.uniform_slots(rng, P.N // 2, complex_values=False).real
    cts[0] = encrypt_slots(orc, P, s_ntt, z.astype(np.complex128), scale, level, 12, "gpu/pt/enc")
    out = empty_dev((B, 2, level - depth + 1, P.N))
    s_out = lib.ckks_poly_eval_tree(ctx, to_dev(cts), B, level, scale, coeffs, to_dev(rlk), out)
    got = to_host(out)
    ref, ref_scale = orc.poly_eval_tree(P, level, cts, scale, coeffs, rlk)
    assert s_out == ref_scale == scale
    assert np.array_equal(got, ref)
    fit = np.polynomial.polynomial.polyval(z, coeffs)
    if level - depth == 0 and np.max(np.abs(fit)) >= 0.45:
        return  # one 54-bit limb at scale 2^54 holds values below 1/2 only
    dec = orc.decrypt(P, level - depth, got[0], s_ntt, s_out).real
    # inputs in [-4, 0] taken directly: the high part's absolute noise (about
    # 1e-12 after relinearisations at N = 2^12, h = 192) is multiplied by x^8,
    # up to 65536; with |x| <= 1 every intermediate stays below 1
    tol = 2e-7 if fn == "exp" else 2 ** -28
    assert np.max(np.abs(dec - fit)) < tol
    if fn == "exp":
        assert np.max(np.abs(dec - np.exp(z))) < tol
    if fn == "exp_u":
        assert np.max(np.abs(dec - np.exp(4.0 * z))) < 1e-8


def test_poly_eval_tree_full_size(lib, orc):
    """N = 2^16 with the C3 primes: degree 5 (depth 3) on one ciphertext at
    level 23, every word against the oracle."""
    ctx, P = config_pair(lib, orc, "C3")
    announce("poly_eval_tree N=2^16 degree 5")
    coeffs = [0.5, -1.0, 0.25, 0.125, -0.5, 0.0625]
    rlk = S.uniform_limbs(S.stream(3, "gpu/ptf/k"), P.mods, P.N, lead=(P.dnum, 2))
    cts = S.uniform_limbs(S.stream(3, "gpu/ptf/ct"), P.q, P.N, lead=(1, 2))
    out = empty_dev((1, 2, 24 - lib.tree_depth(5), P.N))
    lib.ckks_poly_eval_tree(ctx, to_dev(cts), 1, 23, 2.0 ** 54, coeffs, to_dev(rlk), out)
    ref, _ = orc.poly_eval_tree(P, 23, cts, 2.0 ** 54, coeffs, rlk)
    assert np.array_equal(to_host(out), ref)


def test_poly_eval_tree_errors(lib, orc, c3small):
    ctx, P = c3small
    x = empty_dev((1, 2, 4, P.N))
    k = empty_dev((3, 2, 32, P.N))
    y = empty_dev((1, 2, 4, P.N))
    for level, coeffs, code in [(3, [1.0] * 10, lib.CKKS_ERANGE),    # degree 9: depth 4 > level 3
                                (3, [1.0], lib.CKKS_ERANGE),         # degree 0
                                (3, [0.5] * 66, lib.CKKS_ERANGE),    # degree 65
                                (3, [0.0, 2.0 ** 40], lib.CKKS_EINVAL)]:
        with pytest.raises(lib.CKKSError) as e:
            lib.ckks_poly_eval_tree(ctx, x, 1, level, 2.0 ** 54, coeffs, k, y)
        assert e.value.code == code


# ---------------------------------------------------------------- rescale, multiply

@pytest.mark.parametrize("level", [23, 1])
def test_rescale_parity(lib, orc, c3small, level):
    ctx, P = c3small
    announce("rescale level=%d" % level)
    B = 3
    cts = S.uniform_limbs(S.stream(level, "gpu/rs"), P.q[: level + 1], P.N, lead=(B, 2))
    out = empty_dev((B, 2, level, P.N))
    lib.ckks_rescale(ctx, to_dev(cts), out, B, level)
    got = to_host(out)
    for b in range(B):
        assert np.array_equal(got[b], orc.rescale(P, level, cts[b]))
    with pytest.raises(lib.CKKSError) as e:
        lib.ckks_rescale(ctx, to_dev(cts), out, B, 0)
    assert e.value.code == lib.CKKS_ERANGE


@pytest.mark.parametrize("flags", [0, 2])
def test_mul_relin_rescale_parity(lib, orc, c3small, flags):
    ctx, P = c3small
    level = 23
    B = 5
    announce("mul_relin_rescale flags=%d" % flags)
    a = S.uniform_limbs(S.stream(1, "gpu/mrr/a"), P.q, P.N, lead=(B, 2))
    b = S.uniform_limbs(S.stream(1, "gpu/mrr/b"), P.q, P.N, lead=(B, 2))
    rlk = S.uniform_limbs(S.stream(1, "gpu/mrr/k"), P.mods, P.N, lead=(P.dnum, 2))
    lo = level + 1 if flags else level
    out = empty_dev((B, 2, lo, P.N))
    lib.ckks_mul_relin_rescale(ctx, to_dev(a), to_dev(b), to_dev(rlk), out, B, level, flags)
    assert np.array_equal(to_host(out), orc.mul_relin_rescale(P, level, a, b, rlk, flags))


@pytest.mark.parametrize("shape", [(12, 2, 3, 4, 3), (5, 1, 2, 3, 1), (20, 5, 2, 1, 4), (8, 3, 4, 5, 2),
                                   (6, 1, 2, 2, 9)],
                         ids=lambda s: "l%d_in%d_out%d_n1%d_n2%d" % s)
def test_ptmatvec_parity(lib, orc, c3small, shape):
    """BSGS shapes with partial 8-term groups, a single baby or giant step,
    more than 8 (c, b) terms, and more than 8 giant steps (the kernel that
    keeps the giant-step sums in memory order instead of registers)."""
    ctx, P = c3small
    level, n_in, n_out, n1, n2 = shape
    announce("ptmatvec %s" % (shape,))
    x = S.uniform_limbs(S.stream(4, "gpu/pmv/x"), P.q[: level + 1], P.N, lead=(n_in, 2))
    diags = S.uniform_limbs(S.stream(4, "gpu/pmv/d"), P.q[: level + 1], P.N, lead=(n_out, n_in, n2, n1))
    gb = [P.galois(b) for b in range(1, n1)]
    gg = [P.galois(n1 * g) for g in range(1, n2)]
    kb = [S.uniform_limbs(S.stream(i, "gpu/pmv/kb"), P.mods, P.N, lead=(P.dnum, 2)) for i in range(n1 - 1)]
    kg = [S.uniform_limbs(S.stream(i, "gpu/pmv/kg"), P.mods, P.N, lead=(P.dnum, 2)) for i in range(n2 - 1)]
    for flags in (0, 2):
        lo = level + 1 if flags else level
        y = empty_dev((n_out, 2, lo, P.N))
        lib.ckks_ptmatvec(ctx, to_dev(x), n_in, to_dev(diags), n_out, n1, n2, gb, [to_dev(k) for k in kb], gg,
                          [to_dev(k) for k in kg], y, level, flags)
        ref = orc.ptmatvec(P, level, x, diags, gb, kb, gg, kg, flags)
        assert np.array_equal(to_host(y), ref)


@pytest.mark.parametrize("shape", [(12, 2, 2, 3, 3), (5, 1, 3, 2, 1), (20, 3, 1, 1, 4), (8, 3, 2, 5, 2),
                                   (6, 1, 2, 2, 9)],
                         ids=lambda s: "l%d_in%d_out%d_n1%d_n2%d" % s)
def test_ctmatvec_parity(lib, orc, c3small, shape):
    """Encrypted-weight BSGS: partial 8-term groups, a single baby or giant
    step, 15 terms, 9 giant steps."""
    ctx, P = c3small
    level, n_in, n_out, n1, n2 = shape
    announce("ctmatvec %s" % (shape,))
    x = S.uniform_limbs(S.stream(5, "gpu/cmv/x"), P.q[: level + 1], P.N, lead=(n_in, 2))
    diags = S.uniform_limbs(S.stream(5, "gpu/cmv/d"), P.q[: level + 1], P.N, lead=(n_out, n_in, n2, n1, 2))
    rlk = S.uniform_limbs(S.stream(5, "gpu/cmv/rlk"), P.mods, P.N, lead=(P.dnum, 2))
    gb = [P.galois(b) for b in range(1, n1)]
    gg = [P.galois(n1 * g) for g in range(1, n2)]
    kb = [S.uniform_limbs(S.stream(i, "gpu/cmv/kb"), P.mods, P.N, lead=(P.dnum, 2)) for i in range(n1 - 1)]
    kg = [S.uniform_limbs(S.stream(i, "gpu/cmv/kg"), P.mods, P.N, lead=(P.dnum, 2)) for i in range(n2 - 1)]
    for flags in (0, 2):
        lo = level + 1 if flags else level
        y = empty_dev((n_out, 2, lo, P.N))
        lib.ckks_ctmatvec(ctx, to_dev(x), n_in, to_dev(diags), n_out, n1, n2, to_dev(rlk), gb,
                          [to_dev(k) for k in kb], gg, [to_dev(k) for k in kg], y, level, flags)
        ref = orc.ctmatvec(P, level, x, diags, rlk, gb, kb, gg, kg, flags)
        assert np.array_equal(to_host(y), ref)


def test_ctmatvec_trivial_diagonals_equal_ptmatvec(lib, orc, c3small):
    """Diagonals (pt, 0) through ckks_ctmatvec give ckks_ptmatvec's words."""
    ctx, P = c3small
    level, n_in, n_out, n1, n2 = 9, 2, 2, 4, 2
    announce("ctmatvec trivial diagonals")
    x = S.uniform_limbs(S.stream(6, "gpu/cmv/tx"), P.q[: level + 1], P.N, lead=(n_in, 2))
    pts = S.uniform_limbs(S.stream(6, "gpu/cmv/tp"), P.q[: level + 1], P.N, lead=(n_out, n_in, n2, n1))
    cd = np.zeros((n_out, n_in, n2, n1, 2, level + 1, P.N), dtype=np.uint64)
    cd[:, :, :, :, 0] = pts
    rlk = S.uniform_limbs(S.stream(6, "gpu/cmv/trlk"), P.mods, P.N, lead=(P.dnum, 2))
    gb = [P.galois(b) for b in range(1, n1)]
    gg = [P.galois(n1 * g) for g in range(1, n2)]
    kb = [to_dev(S.uniform_limbs(S.stream(i, "gpu/cmv/tkb"), P.mods, P.N, lead=(P.dnum, 2))) for i in range(n1 - 1)]
    kg = [to_dev(S.uniform_limbs(S.stream(i, "gpu/cmv/tkg"), P.mods, P.N, lead=(P.dnum, 2))) for i in range(n2 - 1)]
    y1 = empty_dev((n_out, 2, level, P.N))
    y2 = empty_dev((n_out, 2, level, P.N))
    lib.ckks_ctmatvec(ctx, to_dev(x), n_in, to_dev(cd), n_out, n1, n2, to_dev(rlk), gb, kb, gg, kg, y1, level)
    lib.ckks_ptmatvec(ctx, to_dev(x), n_in, to_dev(pts), n_out, n1, n2, gb, kb, gg, kg, y2, level)
    assert np.array_equal(to_host(y1), to_host(y2))


def _fuzz_cases(n=10, seed=2025):
    """Random parameter sets; every other case sits at a level in the upper
    half of its range (at least L/2), where more digits are active."""
    rng = np.random.default_rng(seed)
    cases = []
    for i in range(n):
        log_n = int(rng.integers(10, 14))
        L = int(rng.integers(2, 17))
        dnum = int(rng.integers(1, min(L, 4) + 1))
        K = -(-L // dnum)
        q_bits = int(rng.choice([30, 40, 54, 55, 56, 57, 59]))
        p_bits = int(rng.choice([min(q_bits + 6, 60), 60]))
        level = int(rng.integers(L // 2, L)) if i % 2 == 0 else int(rng.integers(0, L))
        batch = int(rng.integers(1, 7))
        ks = [int(k) for k in rng.integers(0, 1 << (log_n - 1), size=batch)]
        acc = int(rng.integers(0, 2))
        cases.append((log_n, L, q_bits, K, p_bits, dnum, level, tuple(ks), acc))
    return cases


@pytest.mark.parametrize("case", _fuzz_cases(), ids=lambda c: "logn%d_L%d_q%d_K%d_dnum%d_l%d_b%d" % (
    c[0], c[1], c[2], c[3], c[5], c[6], len(c[7])))
def test_rotate_fuzz(lib, orc, case):
    """Seeded random parameter sets (30- to 59-bit ciphertext primes, special
    primes of 36 to 60 bits, 1 to 4 digits), levels (half of them in the
    upper half of the range), offsets and the accumulate flag: words equal the
    oracle's."""
    log_n, L, q_bits, K, p_bits, dnum, level, ks, acc = case
    announce("rotate fuzz %s" % (case,))
    ctx, P = make_pair(lib, orc, log_n, L, q_bits, K, p_bits, dnum)
    B = len(ks)
    cts = S.uniform_limbs(S.stream(log_n * 100 + L, "gpu/fuzz/ct"), P.q[: level + 1], P.N, lead=(B, 2))
    gs = [P.galois(k) for k in ks]
    keys = [S.uniform_limbs(S.stream(b, "gpu/fuzz/k"), P.mods, P.N, lead=(P.dnum, 2)) for b in range(B)]
    out = empty_dev(cts.shape)
    flags = lib.CKKS_ROT_ACCUMULATE if acc else 0
    lib.ckks_rotate(ctx, to_dev(cts), out, B, level, gs, [to_dev(k) for k in keys], flags)
    ref = orc.rotate_batch(P, level, cts, gs, keys, orc.ROT_ACCUMULATE if acc else 0)
    assert np.array_equal(to_host(out), ref)
    ctx.close()


def test_matvec_errors(lib, orc, c3small):
    """Both BSGS products reject bad arguments on the host, before any launch."""
    ctx, P = c3small
    x = empty_dev((1, 2, 24, P.N))
    k = empty_dev((3, 2, 32, P.N))
    pd = empty_dev((1, 1, 2, 2, 24, P.N))
    cd = empty_dev((1, 1, 2, 2, 2, 24, P.N))
    y = empty_dev((1, 2, 24, P.N))
    g5, g25 = P.galois(1), P.galois(2)
    cases = [  # (n_in, level, baby g, giant g, baby keys, flags, code)
        (1, 24, [g5], [g25], [k], 0, lib.CKKS_ERANGE),
        (1, 0, [g5], [g25], [k], 0, lib.CKKS_ERANGE),
        (1, 23, [g5], [g25], [k], 4, lib.CKKS_EINVAL),
        (1, 23, [6], [g25], [k], 0, lib.CKKS_EINVAL),
        (0, 23, [g5], [g25], [k], 0, lib.CKKS_EINVAL),
    ]
    for n_in, level, gb, gg, kb, flags, code in cases:
        with pytest.raises(lib.CKKSError) as e:
            lib.ckks_ptmatvec(ctx, x, n_in, pd, 1, 2, 2, gb, kb, gg, [k], y, level, flags)
        assert e.value.code == code
        with pytest.raises(lib.CKKSError) as e:
            lib.ckks_ctmatvec(ctx, x, n_in, cd, 1, 2, 2, k, gb, kb, gg, [k], y, level, flags)
        assert e.value.code == code
    with pytest.raises(lib.CKKSError) as e:
        lib.ckks_ptmatvec(ctx, x, 1, misaligned_dev(pd.shape), 1, 2, 2, [g5], [k], [g25], [k], y, 23)
    assert e.value.code == lib.CKKS_EINVAL
    with pytest.raises(lib.CKKSError) as e:
        lib.ckks_ctmatvec(ctx, x, 1, cd, 1, 2, 2, misaligned_dev(k.shape), [g5], [k], [g25], [k], y, 23)
    assert e.value.code == lib.CKKS_EINVAL
    for f in (lib.ckks_ptmatvec, ):  # a missing key is caught by the binding
        with pytest.raises(lib.ArgumentError):
            f(ctx, x, 1, pd, 1, 2, 2, [g5], [None], [g25], [k], y, 23)


def test_empty_batches(lib, orc, c3small):
    """Batch 0 is a no-op for every batched call: no error, output untouched."""
    ctx, P = c3small
    torch = torch_cuda()
    x = empty_dev((1, 2, 24, P.N))
    k = empty_dev((3, 2, 32, P.N))
    y = torch.full((1, 2, 24, P.N), 7, dtype=torch.int64, device="cuda")
    lib.ckks_rotate(ctx, x, y, 0, 23, [], [])
    lib.ckks_rescale(ctx, x, y, 0, 23)
    lib.ckks_mul_relin_rescale(ctx, x, x, k, y, 0, 23)
    lib.ckks_poly_eval(ctx, x, 0, 23, 2.0 ** 54, [0.5, 1.0], k, y)
    lib.ckks_poly_eval_tree(ctx, x, 0, 23, 2.0 ** 54, [0.5, 1.0, 0.25], k, y)
    torch.cuda.synchronize()
    assert bool((y == 7).all())


def test_repeatable(lib, orc, c3small):
    """Same call twice gives identical words (no races between tiles)."""
    ctx, P = c3small
    level = 23
    announce("repeatable")
    cts = S.uniform_limbs(S.stream(9, "gpu/rep"), P.q, P.N, lead=(4, 2))
    keys = [to_dev(S.uniform_limbs(S.stream(b, "gpu/rep/k"), P.mods, P.N, lead=(P.dnum, 2))) for b in range(4)]
    gs = [P.galois(k) for k in (1, 2, 3, 4)]
    d = to_dev(cts)
    o1, o2 = empty_dev(cts.shape), empty_dev(cts.shape)
    lib.ckks_rotate(ctx, d, o1, 4, level, gs, keys)
    lib.ckks_rotate(ctx, d, o2, 4, level, gs, keys)
    assert np.array_equal(to_host(o1), to_host(o2))


# Key switches that raise more limbs than one launch of transforms lists
# (160), on every call that raises digits by the two passes: 14 digits of one
# limb (196 transforms at the top level), 8 digits of 5 (320, two full
# launches), 64 digits of one (4096), and a ring past the one-workgroup
# transforms' limit.
MANY_TRANSFORMS = [
    # log_n, L, q_bits, K, p_bits, dnum, levels
    (10, 14, 50, 1, 60, 14, (13, 12)),
    (10, 40, 50, 5, 60, 8, (39, 28)),
    (10, 64, 54, 1, 60, 64, (63,)),
    (13, 14, 54, 1, 60, 14, (13,)),
]


@pytest.mark.parametrize("shape", MANY_TRANSFORMS, ids=lambda s: "logn%d_L%d_K%d_dnum%d" % (s[0], s[1], s[3], s[5]))
def test_more_transforms_than_a_launch_lists(lib, orc, shape):
    log_n, L, q_bits, K, p_bits, dnum, levels = shape
    ctx, P = make_pair(lib, orc, log_n, L, q_bits, K, p_bits, dnum)
    keys = [S.uniform_limbs(S.stream(b, "gpu/many/k"), P.mods, P.N, lead=(P.dnum, 2)) for b in range(2)]
    d_keys = [to_dev(k) for k in keys]
    gs = [P.galois(1), P.galois(P.N // 2 - 5)]
    for level in levels:
        nq = level + 1
        assert P.beta(level) * (nq + K) - nq > 160
        announce("many transforms %s level=%d" % (shape[:6], level))
        ct = S.uniform_limbs(S.stream(level, "gpu/many/ct"), P.q[:nq], P.N, lead=(2, 2))
        d_ct = to_dev(ct)
        out = empty_dev((2, nq, P.N))
        lib.ckks_keyswitch(ctx, d_ct[0, 1].contiguous(), d_keys[0], out, level)
        assert np.array_equal(to_host(out), orc.keyswitch(P, level, ct[0, 1], keys[0])), "keyswitch"
        out = empty_dev(ct.shape)
        lib.ckks_rotate(ctx, d_ct, out, 2, level, gs, d_keys)
        assert np.array_equal(to_host(out), orc.rotate_batch(P, level, ct, gs, keys)), "rotate"
        out = empty_dev((1, 2) + ct.shape[1:])
        lib.ckks_rotate_hoisted(ctx, d_ct[:1].contiguous(), 1, level, gs, d_keys, out)
        assert np.array_equal(to_host(out)[0], orc.rotate_hoisted(P, level, ct[0], gs, keys)), "hoisted"
        out = empty_dev((1, 2, level, P.N))
        lib.ckks_mul_relin_rescale(ctx, d_ct[:1].contiguous(), d_ct[1:].contiguous(), d_keys[0], out, 1, level)
        assert np.array_equal(to_host(out), orc.mul_relin_rescale(P, level, ct[:1], ct[1:], keys[0])), "product"
        out = empty_dev(ct.shape)
        lib.ckks_rotate_sum(ctx, d_ct, out, 2, level, lib.RotateSum([gs], [d_keys]))
        for b in range(2):
            assert np.array_equal(to_host(out)[b], orc.rotate_sum(P, level, ct[b], [gs], [keys])), "sum"
        out = empty_dev((1, 1, 1, 2, level, P.N))
        lib.ckks_attn_scores(ctx, d_ct[:1].contiguous(), 1, d_ct[1:].contiguous(), 1, 1, level, d_keys[0], None, out)
        ref = orc.attn_scores(P, level, ct[None, :1], ct[None, 1:], keys[0], [], [])
        assert np.array_equal(to_host(out), ref), "scores"
    ctx.close()
