"""Every tile of the product with an 8-bit matrix, whole and ragged, in every
number of digits, against the oracle word for word: plain sums with a bias,
scales on the outputs and on the inputs, each without and with a token row.
tests/test_linear_tiles.py checks that the shapes reach the kernels they are meant for."""
import pytest

from gpu_util import announce, make_pair, torch_cuda
from linear_tiles import CASES, DIGITS, SHAPES, edges
from test_gpu_linear import matmul

pytestmark = pytest.mark.gpu

FORMS = [("none", 0, True), ("none", 1, True), ("out", 0, True), ("out", 1, True), ("in", 0, True), ("in", 1, False)]


@pytest.fixture(scope="module")
def lib():
    torch_cuda()
    import private_rns_ckks_amd as L

    return L


@pytest.fixture(scope="module")
def sets(lib, orc):
    made = {}

    def get(bits):
        if bits not in made:
            made[bits] = make_pair(lib, orc, 10, 3, bits, 0, 60, 1)
        return made[bits]

    yield get
    for ctx, _ in made.values():
        ctx.close()


@pytest.mark.parametrize("bits,rows,n_in,n_out", CASES)
def test_tile(lib, orc, sets, bits, rows, n_in, n_out):
    ctx, P = sets(bits)
    several = (n_in, n_out) != SHAPES[rows][0]
    for k, (scales, tok, bias) in enumerate(FORMS):
        announce("%d digits, tile of %d, %dx%d, %s tok=%d" % (DIGITS[bits], rows, n_in, n_out, scales, tok))
        top = k % 2 == several  # the largest words and bytes in every form, at one size or the other
        matmul(lib, orc, ctx, P, 2, 1 if several else 2, n_in, n_out, scales, tok, bias, k % 2 == 1, top,
               "extreme" if top else "normal", seed=n_out, check=edges(rows, n_out))
