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
    "nokey": (11, 4, 50, 0, 60, 4),
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
    ("nokey", 3, 1, 19, 12, "out", 1, True, False), ("nokey", 1, 2, 4, 3, "in", 0, True, True),
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
    ("mid", 7, 4, 2, 19), ("small", 6, 4, 1, 70), ("small", 5, 3, 2, 16),  # sums in segments of features, and whole
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
    ("small", 5, 6, 6, 1, 37, [], True), ("mid", 6, 7, 6, 2, 11, [], True), ("q56", 5, 5, 5, 1, 16, [], False),
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


# ---------------------------------------------------------------- together, as they are used

class Calls:
    """One call of each kind on random words of a set, with the oracle's results: `run()` makes them on `ctx`."""

    def __init__(self, lib, orc, P, seed, level=6, B=2, F=5, n_out=20, n_in=18):
        self.lib, self.P, self.level, self.B, self.F, self.n_in, self.n_out = lib, P, level, B, F, n_in, n_out
        self.st, (gal, keys) = steps(lib, P, [2], seed=8)
        rlk, lv, N = key(P, 8, "rlk"), level, P.N
        rng = S.stream(8, "linear/calls")
        self.w, self.sc = matrix(8, n_out, n_in), np.exp(rng.normal(-4, 0.3, n_out))
        self.gamma, self.beta, self.bias = rng.normal(1, 0.5, F), rng.normal(0, 1, F), rng.normal(0, 1, n_out)
        self.scale = 2.0 ** 37
        self.host = self.inputs(seed)
        self.dev = {k: to_dev(v) for k, v in self.host.items()}
        self.d_w, self.d_rlk = int8_dev(self.w), to_dev(rlk)
        self.out = {"y": empty_dev((B, n_out, 2, lv - 1, N)), "sum": empty_dev((B, 2, lv + 1, N)),
                    "var": empty_dev((B, 2, lv - 1, N)), "norm": empty_dev((B, F, 2, lv - 3, N)),
                    "dx": empty_dev((B, F, 2, lv - 4, N)), "dgamma": empty_dev((F, 2, lv, N)),
                    "dbeta": empty_dev((F, 2, lv + 1, N))}

        def ref(h):
            r = {"y": orc.matmul_i8(P, lv, h["x"], self.w, self.scale, self.sc, False, h["tok"], self.scale, self.bias)[0]}
            r["sum"], r["var"] = orc.layernorm_var(P, lv, h["f"], self.scale, 0.5, rlk)
            low = np.ascontiguousarray(h["r"][..., :lv - 1, :])
            r["norm"] = orc.layernorm(P, h["f"], r["sum"], low, self.scale, self.scale, self.gamma, self.beta, rlk)
            r.update(orc.layernorm_grad(P, lv, h["f"], h["xh"], h["r"], self.scale, self.scale, self.gamma, rlk, gal, keys))
            return r

        self.ref = ref

    def inputs(self, seed):
        P, n, B, F = self.P, self.level + 1, self.B, self.F
        h = {"x": words(P, seed, "cx", n, (B, self.n_in, 2)), "tok": words(P, seed, "ct", n, (1,)),
             "f": words(P, seed, "cf", n, (B, F, 2)), "xh": words(P, seed, "ch", n, (B, F, 2)),
             "r": words(P, seed, "cr", n, (B, 2))}
        h["low"] = np.ascontiguousarray(h["r"][..., :n - 2, :])
        return h

    def set(self, seed):
        self.host = self.inputs(seed)
        for k, v in self.host.items():
            self.dev[k].copy_(to_dev(v))

    def run(self, ctx, only=("matmul", "var", "norm", "grad"), stream=None):
        lib, d, o, lv, B, F = self.lib, self.dev, self.out, self.level, self.B, self.F
        if "matmul" in only:
            lib.ckks_matmul_i8(ctx, d["x"], B, self.n_in, self.d_w, self.n_out, lv, self.scale, o["y"], scales=self.sc,
                               d_tok=d["tok"], n_tok=1, tok_scale=self.scale, bias=self.bias, stream=stream)
        if "var" in only:
            lib.ckks_layernorm_var(ctx, d["f"], B, F, lv, self.scale, 0.5, self.d_rlk, o["sum"], o["var"], stream=stream)
        if "norm" in only:
            lib.ckks_layernorm(ctx, d["f"], o["sum"], B, F, lv, self.scale, d["low"], lv - 2, self.scale, self.gamma,
                               self.beta, self.d_rlk, o["norm"], stream=stream)
        if "grad" in only:
            lib.ckks_layernorm_grad(ctx, d["f"], B, F, lv, d["xh"], lv, self.scale, d["r"], lv, self.scale, self.gamma,
                                    self.d_rlk, self.st, d_dx=o["dx"], d_dgamma=o["dgamma"], d_dbeta=o["dbeta"],
                                    stream=stream)

    def clear(self):
        for t in self.out.values():
            t.zero_()

    def check(self, what=""):
        for k, v in self.ref(self.host).items():
            same(self.out[k], v, what + " " + k)


def test_on_another_stream_and_in_a_row(lib, orc, sets):
    """Calls in a row on a side stream, which read what that stream writes only after long work of its own."""
    torch = torch_cuda()
    ctx, P = sets("small")
    announce("side stream, late inputs")
    c = Calls(lib, orc, P, 1)
    src = {k: v.clone() for k, v in c.dev.items()}
    for v in c.dev.values():
        v.zero_()
    c.run(ctx)  # sizes the context's buffers
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn(3000, 3000, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(10):
            busy = busy @ busy * 1e-4
        for k, v in src.items():
            c.dev[k].copy_(v)
        c.run(ctx)  # the current stream
    side.synchronize()
    c.check("late")
    c.clear()
    torch.cuda.synchronize()
    c.run(ctx, stream=side)
    side.synchronize()
    c.check("by argument")


@pytest.mark.parametrize("op", ["matmul", "var", "norm", "grad"])
def test_captured_calls_replay(lib, orc, op):
    """A call captured after an eager one: every replay equals the oracle's words on new inputs, with eager calls
    of the same context between the replays and after a larger call has grown its buffers.  A first call that
    would have to allocate raises and leaves the capture usable."""
    torch = torch_cuda()
    ctx, P = make_pair(lib, orc, *SETS["small"])
    announce("captured " + op)
    c = Calls(lib, orc, P, 2)
    if op == "norm":
        c.run(make_pair(lib, orc, *SETS["small"])[0], ("var",))  # its sums, from another context
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    marker = torch.zeros(8, device="cuda")
    with torch.cuda.graph(graph, stream=side):
        with pytest.raises(lib.CKKSError) as e:
            c.run(ctx, (op,))
        marker.add_(1.0)
    assert e.value.code == lib.CKKS_EHIP and "captured" in str(e.value)
    graph.replay()
    torch.cuda.synchronize()
    assert marker.tolist() == [1.0] * 8
    with torch.cuda.stream(side):
        c.run(ctx, (op,))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.run(ctx, (op,))
    names = {"matmul": ["y"], "var": ["sum", "var"], "norm": ["norm"], "grad": ["dx", "dgamma", "dbeta"]}[op]
    other = make_pair(lib, orc, *SETS["small"])[0]
    for i in range(3):
        c.set(20 + i)
        c.clear()
        if op == "norm":
            c.run(other, ("var",))
        graph.replay()
        torch.cuda.synchronize()
        ref = c.ref(c.host)
        for k in names:
            same(c.out[k], ref[k], "replay %d %s" % (i, k))
        if i == 0:  # a larger eager call grows the buffers that the graph was captured on
            big = Calls(lib, orc, P, 3, B=4, F=9, n_out=40, n_in=40)
            big.run(ctx)
            big.check("larger")
        c.clear()
        c.run(ctx, (op,) if op != "norm" else ("var", "norm"))
        for k in names:
            same(c.out[k], ref[k], "eager after replay %d %s" % (i, k))
    del graph
    ctx.close()


@pytest.mark.parametrize("mb", [1, 2])
def test_small_blocks(lib, orc, sets, monkeypatch, mb):
    """Operands in blocks of a limited size: the same words; a call with fewer limbs, blocks or features than an
    earlier one then needs nothing new and can be captured."""
    torch = torch_cuda()
    announce("blocks of %d MiB" % mb)
    monkeypatch.setenv("CKKS_BLOCK_MB", str(mb))
    ctx, P = make_pair(lib, orc, *SETS["small"])
    big = Calls(lib, orc, P, 4, B=3, F=13, n_out=70, n_in=40)
    big.run(ctx)
    big.check()
    side = torch.cuda.Stream()
    for kw in (dict(level=6, B=2, F=13, n_out=70), dict(level=5, B=3, F=4, n_out=33), dict(level=5, B=1, F=2, n_out=9, n_in=3)):
        c = Calls(lib, orc, P, 5, **kw)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.run(ctx)
        graph.replay()
        torch.cuda.synchronize()
        c.check(str(kw))
        del graph
    # one block's outputs in several groups, of a matrix that lies either way round
    matmul(lib, orc, ctx, P, 4, 2, 20, 150, "out", 2, True, True)
    matmul(lib, orc, ctx, P, 4, 70, 3, 2, "in", 1, True, False)
    ctx.close()


def test_two_contexts_on_two_streams(lib, orc, sets):
    torch = torch_cuda()
    announce("two contexts")
    made = []
    for name, seed in (("small", 6), ("q56", 7)):
        ctx, P = make_pair(lib, orc, *SETS[name])
        made.append((ctx, Calls(lib, orc, P, seed), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for ctx, c, s in made:
            c.run(ctx, stream=s)
    torch.cuda.synchronize()
    for ctx, c, _ in made:
        c.check()
        ctx.close()


def test_one_buffer_as_several_operands(lib, orc, sets):
    """The gradient that is its own normalised input, one scale for every block, the sum as rstd."""
    ctx, P = sets("small")
    announce("shared operands")
    B, F, lv = 1, 3, 5
    x, rlk = words(P, 9, "own", lv + 1, (B, F, 2)), key(P, 9, "rlk")
    d_x, d_k = to_dev(x), to_dev(rlk)
    dx = empty_dev((B, F, 2, lv - 4, P.N))
    lib.ckks_layernorm_grad(ctx, d_x, B, F, lv, d_x, lv, 2.0 ** 37, d_x, lv, 2.0 ** 37, None, d_k, None, d_dx=dx)
    ref = orc.layernorm_grad(P, lv, x, x, x[:, 0], 2.0 ** 37, 2.0 ** 37, None, rlk, [], [], ("dx",))
    same(dx, ref["dx"])
    s, y = to_dev(x[:, 0]), empty_dev((B, F, 2, lv - 1, P.N))
    lib.ckks_layernorm(ctx, d_x, s, B, F, lv, 2.0 ** 37, s, lv, 2.0 ** 37, None, None, d_k, y)
    same(y, orc.layernorm(P, x, x[:, 0], x[:, 0], 2.0 ** 37, 2.0 ** 37, None, None, rlk))


def test_bytes_outside_the_outputs_stay(lib, orc, sets):
    """Outputs inside larger buffers, ragged tiles among them: the words before and behind are left as they were."""
    torch = torch_cuda()
    ctx, P = sets("small")
    announce("guard words")
    c = Calls(lib, orc, P, 10, n_out=33, n_in=17)
    N, whole = P.N, {}
    for k, t in c.out.items():
        buf = torch.full((t.numel() + 4 * N,), -7, dtype=torch.int64, device="cuda")
        whole[k], c.out[k] = buf, buf[2 * N:2 * N + t.numel()].view(t.shape)
    c.run(ctx)
    c.check()
    for k, buf in whole.items():
        h = to_host(buf).view(np.int64)
        assert (h[:2 * N] == -7).all() and (h[-2 * N:] == -7).all(), k


def test_zero_rows_and_gradients(lib, orc, sets):
    """A token row of zeros, a matrix of zeros, gamma of zero and gradients of zero: the words the oracle has."""
    ctx, P = sets("small")
    announce("zeros")
    B, n_in, n_out, lv = 2, 20, 9, 4
    x, tok = words(P, 11, "zx", lv + 1, (B, n_in, 2)), words(P, 11, "zt", lv + 1, (2,))
    tok[1] = 0
    out = empty_dev((B, n_out, 2, lv, P.N))
    for w in (matrix(11, n_out, n_in), np.zeros((n_out, n_in), np.int8)):
        lib.ckks_matmul_i8(ctx, to_dev(x), B, n_in, int8_dev(w), n_out, lv, 2.0 ** 37, out, d_tok=to_dev(tok), n_tok=2,
                           tok_scale=2.0 ** 37, bias=np.ones(n_out))
        ref, _ = orc.matmul_i8(P, lv, x, w, 2.0 ** 37, None, False, tok, 2.0 ** 37, np.ones(n_out))
        same(out, ref)
        assert (to_host(out)[1, :, 1] == 0).all()  # nothing but the bias is left of the second block
    F, rlk = 3, key(P, 11, "rlk")
    dy, xh, r = np.zeros((1, F, 2, 6, P.N), np.uint64), words(P, 11, "zh", 6, (1, F, 2)), words(P, 11, "zr", 6, (1, 2))
    dx, dg, db = empty_dev((1, F, 2, 1, P.N)), empty_dev((F, 2, 5, P.N)), empty_dev((F, 2, 6, P.N))
    lib.ckks_layernorm_grad(ctx, to_dev(dy), 1, F, 5, to_dev(xh), 5, 2.0 ** 37, to_dev(r), 5, 2.0 ** 37, np.zeros(F),
                            to_dev(rlk), None, dx, dg, db)
    for t in (dx, dg, db):
        assert (to_host(t) == 0).all()


def test_as_many_inputs_as_allowed(lib, orc, sets):
    """65536 inputs at the top of the range against -128 and 127 everywhere: sums of bytes come within a factor of
    two of 2^31."""
    announce("65536 inputs")
    ctx, P = make_pair(lib, orc, 10, 1, 54, 0, 60, 1)
    matmul(lib, orc, ctx, P, 0, 1, 65536, 9, "none", 0, False, False, True, "extreme", check=[0, 4, 8])
    matmul(lib, orc, ctx, P, 0, 1, 65536, 2, "none", 0, False, False, True, "extreme")
    ctx.close()


MIXED = {"narrow": ([54, 30, 47, 56, 40, 59, 24], [60, 60, 59], 3), "wide": ([62, 30, 54, 61, 24, 60, 45], [62, 61, 60], 3)}


@pytest.mark.parametrize("name", list(MIXED))
@pytest.mark.parametrize("top", [False, True])
def test_primes_of_several_sizes(lib, orc, name, top):
    """One basis with primes of 24 to 62 bits: quotients and bytes go by each limb's prime, digits by the largest."""
    announce("mixed primes %s" % name)
    bits, p_bits, dnum = MIXED[name]
    seen, q = {}, []
    for b in bits + p_bits:
        seen[b] = seen.get(b, 0) + 1
        q.append(lib.ckks_find_primes(10, b, seen[b])[-1])
    q, p = q[:len(bits)], q[len(bits):]
    ctx, P = lib.Context(10, q, p, dnum), orc.Params(10, q, p, dnum)
    for args in ((5, 1, 40, 12, "out", 1), (3, 2, 17, 140, "in", 0), (6, 1, 5, 3, "none", 0)):
        matmul(lib, orc, ctx, P, *args, top=top, kind="extreme" if top else "normal")
    c = Calls(lib, orc, P, 12)
    c.scale = 2.0 ** 25
    c.run(ctx)
    c.check()
    ctx.close()


@pytest.mark.parametrize("op", ["matmul", "norm"])
def test_full_ring(lib, orc, sets, op):
    """N = 2^16, the shape the calls are used at."""
    ctx, P = sets("full")
    announce("full ring " + op)
    if op == "matmul":
        matmul(lib, orc, ctx, P, 2, 1, 24, 130, "out", 0, True, check=[0, 63, 64, 127, 128, 129])
        matmul(lib, orc, ctx, P, 3, 1, 33, 20, "in", 1, True, True, check=[0, 7, 19])
        matmul(lib, orc, ctx, P, 2, 1, 9, 2, "none", 1, True)
        return
    c = Calls(lib, orc, P, 13, level=5, B=1, F=3)
    c.scale = 2.0 ** 51
    c.run(ctx, ("var", "norm", "grad"))
    ref = c.ref(c.host)
    for k in ("sum", "var", "norm", "dx", "dgamma", "dbeta"):
        same(c.out[k], ref[k], k)


def test_traced_families(lib, orc, sets):
    ctx, P = sets("small")
    announce("traced families")
    c = Calls(lib, orc, P, 14)
    counts = {}
    for family in ("matmul_i8", "layernorm"):
        lib.ckks_trace_begin(ctx, family)
        c.run(ctx)
        t = lib.ckks_trace_end(ctx)
        counts[family] = t["launches"]
        assert t["work_units"] > 0
    assert counts == {"matmul_i8": 1, "layernorm": 6}


def test_block_forwards_and_backwards_encrypted(lib, orc):
    """A layer norm whose weight and bias enter the layer behind it, GELU, and the layer after: forwards, and the
    gradients back through the first layer and the norm, on encryptions, word for word as the oracle and decrypting
    to float64 (the tolerance is tests/test_oracle_linear.py's: the products here multiply errors by no more)."""
    torch = torch_cuda()
    from linear_util import features, norm_backward, norm_forward, rsqrt_poly

    tol, lv, F, H, eps, pad = 2.0 ** -20, 16, 6, 20, 1e-3, 5
    ctx, P = make_pair(lib, orc, 10, 17, 50, 6, 60, 3)
    announce("encrypted block")
    s, s_ntt = secret(orc, P, 15, 64)
    rlk, scale, n = relin_key(orc, P, s_ntt, 15), 2.0 ** 50, P.N // 2
    rng = S.stream(15, "linear/block")
    coeffs, _ = rsqrt_poly(0.4)
    x = features(rng, F, n, pad, 0.4, eps)
    gamma, beta = rng.uniform(0.5, 1.5, F), rng.normal(0, 0.3, F)
    w1, w2 = matrix(16, H, F), matrix(17, F, H)
    s1, s2 = 0.004, rng.uniform(0.002, 0.004, F)
    enc = lambda z, l, t: encrypt_slots(orc, P, s_ntt, z.astype(np.complex128), scale, l, 15, t)
    dec = lambda ct, sc: orc.decrypt(P, ct.shape[-2] - 1, ct, s_ntt, sc).real
    err = lambda got, ref: float(np.max(np.abs(got - ref)) / np.max(np.abs(ref)))
    d_k = to_dev(rlk)
    ct = np.stack([enc(v, lv, "x%d" % i) for i, v in enumerate(x)])[None]
    d_x, d_sum, d_u = to_dev(ct), empty_dev((1, 2, lv + 1, P.N)), empty_dev((1, 2, lv - 1, P.N))
    lib.ckks_layernorm_var(ctx, d_x, 1, F, lv, scale, eps - 1, d_k, d_sum, d_u)
    d_r = empty_dev((1, 2, lv - 4, P.N))
    s_r = lib.ckks_poly_eval_tree(ctx, d_u, 1, lv - 2, scale, coeffs, d_k, d_r)
    d_h = empty_dev((1, F, 2, lv - 6, P.N))
    lib.ckks_layernorm(ctx, d_x, d_sum, 1, F, lv, scale, d_r, lv - 5, s_r, None, None, d_k, d_h)
    # w1 s1 (gamma xhat + beta): gamma s1 on the inputs, w1 s1 beta in the bias
    l1 = lv - 7
    d_z = empty_dev((1, H, 2, l1, P.N))
    s_z = lib.ckks_matmul_i8(ctx, d_h, 1, F, int8_dev(w1), H, l1, scale, d_z, scales=gamma * s1, bias=s1 * (w1 @ beta),
                             flags=lib.CKKS_SCALE_IN)
    act = [0.0, 0.5, 0.39, 0.0]  # x / 2 + 0.39 x^2, a square-law GELU
    act[3] = 0.01
    d_a = empty_dev((H, 2, l1 - 2, P.N))
    s_a = lib.ckks_poly_eval_tree(ctx, d_z.view(H, 2, l1, P.N), H, l1 - 1, s_z, act, d_k, d_a)
    d_y = empty_dev((1, F, 2, l1 - 3, P.N))
    s_y = lib.ckks_matmul_i8(ctx, d_a, 1, H, int8_dev(w2), F, l1 - 3, s_a, d_y, scales=s2)
    # the oracle's words
    sm, u = orc.layernorm_var(P, lv, ct, scale, eps - 1, rlk)
    same(d_u, u)
    r, s_ro = orc.poly_eval_tree(P, lv - 2, u, scale, coeffs, rlk)
    h = orc.layernorm(P, ct, sm, r, scale, s_r, None, None, rlk)
    z, s_zo = orc.matmul_i8(P, l1, h, w1, scale, gamma * s1, True, None, 1.0, s1 * (w1 @ beta))
    a, s_ao = orc.poly_eval_tree(P, l1 - 1, z[0], s_z, act, rlk)
    y, s_yo = orc.matmul_i8(P, l1 - 3, a[None], w2, s_a, s2)
    assert (s_r, s_z, s_a, s_y) == (s_ro, s_zo, s_ao, s_yo)
    same(d_r, r)
    same(d_h, h)
    same(d_z, z)
    same(d_a, a)
    same(d_y, y)
    # float64
    ref_r = np.polynomial.polynomial.polyval(x.var(0) + eps - 1, coeffs)
    ref_h = norm_forward(x, ref_r)
    ref_z = s1 * (w1 @ (gamma[:, None] * ref_h + beta[:, None]))
    ref_y = s2[:, None] * (w2 @ np.polynomial.polynomial.polyval(ref_z, act))
    for j in range(H):
        assert err(dec(z[0, j], s_z), ref_z[j]) < tol
    for i in range(F):
        assert err(dec(y[0, i], s_y), ref_y[i]) < tol
    # backwards from gradients of z: through w1 (transposed, one scale for every input), then the norm
    lb = l1
    gz = rng.uniform(-1, 1, (H, n)) * (np.arange(n) < n - pad)
    gct = np.stack([enc(v, lb, "g%d" % i) for i, v in enumerate(gz)])[None]
    d_g, d_dx = empty_dev((1, F, 2, lb, P.N)), empty_dev((1, F, 2, lb - 5, P.N))
    s_g = lib.ckks_matmul_i8(ctx, to_dev(gct), 1, H, int8_dev(w1), F, lb, scale, d_g, scales=np.full(H, s1),
                             flags=lib.CKKS_W_TRANSPOSED | lib.CKKS_SCALE_IN)
    lib.ckks_layernorm_grad(ctx, d_g, 1, F, lb - 1, d_h, l1, scale, d_r, lv - 5, s_r, gamma, d_k, None, d_dx=d_dx)
    g, s_go = orc.matmul_i8(P, lb, gct, w1.T, scale, np.full(H, s1), True)
    assert s_g == s_go
    same(d_g, g)
    dx = orc.layernorm_grad(P, lb - 1, g, h, r, scale, s_r, gamma, rlk, [], [], ("dx",))["dx"]
    same(d_dx, dx)
    ref_dx, _ = norm_backward(s1 * (w1.T @ gz), ref_h, ref_r, gamma)
    for i in range(F):
        assert err(dec(dx[0, i], s_g), ref_dx[i]) < tol
    ctx.close()


# ---------------------------------------------------------------- refusals

def test_refusals(lib, orc, sets):
    ctx, P = sets("small")
    announce("refusals")
    E, R = lib.CKKS_EINVAL, lib.CKKS_ERANGE
    c = Calls(lib, orc, P, 16)
    d, o, lv, B, F, N = c.dev, c.out, c.level, c.B, c.F, P.N

    def raises(code, fn, *a, **kw):
        with pytest.raises(lib.CKKSError) as e:
            fn(ctx, *a, **kw)
        assert e.value.code == code, str(e.value)

    big = empty_dev((B, c.n_out, 2, lv + 1, N))

    def mm(code, x=d["x"], B=B, n_in=c.n_in, w=c.d_w, n_out=c.n_out, lv=lv, scale=1.0, y=big, **kw):
        raises(code, lib.ckks_matmul_i8, x, B, n_in, w, n_out, lv, scale, y, **kw)

    mm(E, B=-1)
    mm(E, n_in=0)
    mm(E, n_out=-1)
    mm(R, lv=-1)
    mm(R, lv=P.L)
    mm(R, lv=0, scales=c.sc)
    mm(R, lv=1, scales=c.sc, d_tok=d["tok"], n_tok=1)
    mm(E, flags=16)
    mm(E, flags=lib.CKKS_SCALE_IN)
    mm(E, d_tok=d["tok"], n_tok=0)
    mm(E, d_tok=d["tok"], n_tok=-1)
    mm(E, n_tok=1)
    mm(E, scales=np.full(c.n_out, 2.0 ** 23))  # times a 40-bit prime
    mm(E, scales=np.full(c.n_out, np.nan))
    mm(E, bias=np.full(c.n_out, np.inf))
    mm(E, scale=2.0 ** 61, bias=np.full(c.n_out, 4.0))
    mm(E, x=big)  # an output that overlaps the input
    mis = misaligned_dev((B, c.n_out, 2, lv + 1, N))
    mm(E, y=mis)
    for bad in (dict(w=d["x"]), dict(w=c.d_w[:, ::2]), dict(w=c.d_w[:3]), dict(scales=c.sc[:-1]), dict(bias=c.bias[1:]),
                dict(scales=c.sc, flags=lib.CKKS_SCALE_IN), dict(y=o["sum"]), dict(x=d["f"])):
        with pytest.raises(lib.ArgumentError):
            mm(0, **bad)

    def var(code, x=d["f"], B=B, F=F, lv=lv, scale=c.scale, eps=0.5, rlk=c.d_rlk, s=o["sum"], v=o["var"]):
        raises(code, lib.ckks_layernorm_var, x, B, F, lv, scale, eps, rlk, s, v)

    var(E, B=-1)
    var(E, F=0)
    var(E, F=65537, B=0)
    var(R, lv=1)
    var(R, lv=P.L)
    var(E, scale=0.0)
    var(E, scale=-1.0)
    var(E, scale=float("nan"))
    var(E, scale=2.0 ** 90)  # k rounds to 0
    var(E, scale=1e-30)      # k reaches 2^126
    var(E, eps=float("inf"))
    var(E, s=d["f"])
    var(E, v=c.d_rlk)

    def norm(code, x=d["f"], s=o["sum"], B=B, F=F, lv=lv, scale=c.scale, r=d["low"], t=lv - 2, rs=c.scale, gamma=c.gamma,
             beta=c.beta, y=o["norm"]):
        raises(code, lib.ckks_layernorm, x, s, B, F, lv, scale, r, t, rs, gamma, beta, c.d_rlk, y)

    norm(E, B=-1)
    norm(E, F=0, gamma=None, beta=None)
    norm(R, t=1)
    norm(R, t=lv + 1, lv=lv, r=o["y"])
    norm(E, rs=0.0)
    norm(E, scale=float("inf"))
    norm(E, rs=2.0 ** 100)
    norm(E, gamma=np.full(F, np.nan))
    norm(E, gamma=np.full(F, 1e30))
    norm(E, beta=np.full(F, 1e30))
    norm(E, y=d["f"])
    with pytest.raises(lib.ArgumentError):
        norm(0, gamma=c.gamma[1:])

    def grad(code, dy=d["f"], B=B, F=F, lv=lv, xh=d["xh"], lx=lv, xs=c.scale, r=d["r"], lr=lv, rs=c.scale, gamma=c.gamma,
             st=c.st, dx=o["dx"], dg=o["dgamma"], db=o["dbeta"]):
        raises(code, lib.ckks_layernorm_grad, dy, B, F, lv, xh, lx, xs, r, lr, rs, gamma, c.d_rlk, st, dx, dg, db)

    grad(E, B=-1)
    grad(E, F=0, gamma=None)
    grad(E, dx=None, dg=None, db=None)
    grad(R, lv=4)
    grad(R, lv=0, dx=None)
    grad(R, lx=lv - 1)
    grad(R, lr=lv - 1)
    grad(R, lx=P.L)
    grad(E, xs=0.0)
    grad(E, rs=float("nan"))
    grad(E, xs=2.0 ** 100)
    grad(E, gamma=np.full(F, 1e40))
    grad(E, dx=d["f"])
    grad(E, dg=o["dbeta"])
    bad = lib.RotateSum([[1]], [[c.d_rlk]])
    grad(E, st=bad)
    none = make_pair(lib, orc, 10, 7, 40, 0, 60, 7)[0]  # no special primes
    k = empty_dev((7, 2, 7, N))
    for fn, a in ((lib.ckks_layernorm_var, (d["f"], B, F, lv, c.scale, 0.0, k, o["sum"], o["var"])),
                  (lib.ckks_layernorm, (d["f"], o["sum"], B, F, lv, c.scale, d["low"], lv - 2, c.scale, None, None, k,
                                        o["norm"])),
                  (lib.ckks_layernorm_grad, (d["f"], B, F, lv, d["xh"], lv, c.scale, d["r"], lv, c.scale, None, k, None,
                                             o["dx"]))):
        with pytest.raises(lib.CKKSError) as e:
            fn(none, *a)
        assert e.value.code == lib.CKKS_EPARAM
    none.close()


def test_nothing_to_do(lib, orc, sets):
    """No blocks or no outputs: nothing is written; no blocks leave weights' gradients of zero."""
    torch = torch_cuda()
    ctx, P = sets("small")
    announce("empty calls")
    c = Calls(lib, orc, P, 17)
    for t in c.out.values():
        t.fill_(-7)
    d, o, lv, F = c.dev, c.out, c.level, c.F
    assert lib.ckks_matmul_i8(ctx, d["x"], 0, c.n_in, c.d_w, c.n_out, lv, 3.0, o["y"]) == 3.0
    lib.ckks_matmul_i8(ctx, d["x"], c.B, c.n_in, c.d_w, 0, lv, 3.0, o["y"])
    lib.ckks_layernorm_var(ctx, d["f"], 0, F, lv, c.scale, 0.0, c.d_rlk, o["sum"], o["var"])
    lib.ckks_layernorm(ctx, d["f"], o["sum"], 0, F, lv, c.scale, d["low"], lv - 2, c.scale, None, None, c.d_rlk, o["norm"])
    lib.ckks_layernorm_grad(ctx, d["f"], 0, F, lv, d["xh"], lv, c.scale, d["r"], lv, c.scale, None, c.d_rlk, c.st, o["dx"])
    torch.cuda.synchronize()
    for t in o.values():
        assert bool((t == -7).all())
    lib.ckks_layernorm_grad(ctx, d["f"], 0, F, lv, d["xh"], lv, c.scale, d["r"], lv, c.scale, None, c.d_rlk, c.st, None,
                            o["dgamma"], o["dbeta"])
    torch.cuda.synchronize()
    assert bool((o["dgamma"] == 0).all()) and bool((o["dbeta"] == 0).all())
