"""Where the 8-bit matrix of ckks_matmul_i8 may lie: at any byte, next to the
output but not under it."""
import numpy as np
import pytest

from gpu_util import announce, empty_dev, make_pair, to_dev, torch_cuda
from test_gpu_linear import matrix, same, words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    torch_cuda()
    import private_rns_ckks_amd as L

    return L


@pytest.fixture(scope="module")
def pair(lib, orc):
    ctx, P = make_pair(lib, orc, 10, 2, 50, 0, 60, 1)
    yield ctx, P
    ctx.close()


def at_byte(w, offset):
    """The matrix on the device, `offset` bytes behind a 16-byte boundary."""
    torch = torch_cuda()
    buf = torch.full((w.size + 32,), 77, dtype=torch.int8, device="cuda")
    out = buf[offset:offset + w.size].view(w.shape)
    out.copy_(torch.from_numpy(np.ascontiguousarray(w)))
    assert out.data_ptr() % 16 == offset
    return out


@pytest.mark.parametrize("offset", [1, 6, 8, 15])
@pytest.mark.parametrize("n_in,n_out,transposed", [(5, 3, False), (5, 3, True), (33, 19, False), (33, 19, True)])
def test_matrix_at_any_byte(lib, orc, pair, n_in, n_out, transposed, offset):
    """Rows of a wider matrix, as a device that holds some of the outputs has them."""
    ctx, P = pair
    announce("matrix of %dx%d at byte %d, transposed=%s" % (n_out, n_in, offset, transposed))
    x, w = words(P, 1, "x", 2, (1, n_in, 2)), matrix(1, n_out, n_in)
    y = empty_dev((1, n_out, 2, 2, P.N))
    lib.ckks_matmul_i8(ctx, to_dev(x), 1, n_in, at_byte(w.T if transposed else w, offset), n_out, 1, 2.0 ** 50, y,
                       flags=lib.CKKS_W_TRANSPOSED if transposed else 0)
    same(y, orc.matmul_i8(P, 1, x, w, 2.0 ** 50)[0])


def test_row_slice_of_an_odd_matrix(lib, orc, pair):
    ctx, P = pair
    announce("rows 3..13 of a 20x21 matrix")
    torch = torch_cuda()
    n_in, rows = 21, slice(3, 14)
    x, w = words(P, 2, "x", 2, (2, n_in, 2)), matrix(2, 20, n_in)
    d_w = torch.from_numpy(w).cuda()[rows]
    y = empty_dev((2, 11, 2, 2, P.N))
    lib.ckks_matmul_i8(ctx, to_dev(x), 2, n_in, d_w, 11, 1, 2.0 ** 50, y)
    same(y, orc.matmul_i8(P, 1, x, w[rows], 2.0 ** 50)[0])


@pytest.mark.parametrize("n_in,n_out", [(3, 5), (21, 11)])
def test_matrix_beside_the_output(lib, orc, pair, n_in, n_out):
    """One buffer: the matrix right before the output and right behind it, and one byte into it (refused)."""
    ctx, P = pair
    announce("matrix of %dx%d beside the output" % (n_out, n_in))
    torch = torch_cuda()
    x, w = words(P, 3, "x", 2, (1, n_in, 2)), matrix(3, n_out, n_in)
    d_x, h_w, n = to_dev(x), torch.from_numpy(w).cuda(), n_in * n_out
    ref = orc.matmul_i8(P, 1, x, w, 2.0 ** 50)[0]
    shape, size = (1, n_out, 2, 2, P.N), n_out * 2 * 2 * P.N * 8
    buf = torch.zeros(1024 + size + 1024, dtype=torch.int8, device="cuda")
    y = buf[1024:1024 + size].view(torch.int64).view(shape)

    def call(at):
        d_w = buf[at:at + n].view(n_out, n_in)
        d_w.copy_(h_w)
        lib.ckks_matmul_i8(ctx, d_x, 1, n_in, d_w, n_out, 1, 2.0 ** 50, y)
        same(y, ref, "matrix at byte %d" % at)
        assert torch.equal(d_w, h_w)

    call(1024 - n)
    call(1024 + size)
    for at in (1024 - n + 1, 1024 + size - 1):
        with pytest.raises(lib.CKKSError) as e:
            call(at)
        assert e.value.code == lib.CKKS_EINVAL
