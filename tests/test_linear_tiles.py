"""The rule that picks a product's kernel (csrc/matmul_tiles.h), on the CPU: the
shapes of linear_tiles.py go where they are meant to, and the matrix laid out
for a tile never outgrows its buffer."""
import os
import shutil
import subprocess

import pytest

from linear_tiles import CASES, DIGITS, SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

MAIN = r"""
#include <stdio.h>

#include "matmul_tiles.h"

int main() {
  unsigned long long q;
  int n_in, nj;
  while (scanf("%llu %d %d", &q, &n_in, &nj) == 3) {
    if (!ckks::tiled(n_in, nj)) {
      puts("0 0 0 0 0");
      continue;
    }
    const ckks::Tiles t(n_in, nj);
    printf("%d %d %d %d %llu\n", t.rows(), t.row_blocks, t.chunks, ckks::word_digits(q), (unsigned long long)t.lanes());
  }
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    """[(q, n_in, n_out)] -> [(rows of a tile, tiles, chunks of 32 inputs, digits, lanes of the matrix laid out)]."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    tmp = tmp_path_factory.mktemp("tiles")
    (tmp / "main.cpp").write_text(MAIN)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                           os.path.join(ROOT, "private_rns_ckks_amd", "csrc"), str(tmp / "main.cpp"), "-o", str(tmp / "tiles")])

    def run(items):
        r = subprocess.run([str(tmp / "tiles")], input="".join("%d %d %d\n" % v for v in items), capture_output=True,
                           text=True, timeout=60, check=True)
        return [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]

    return run


def test_every_tile_and_digit_is_reached(rule, orc):
    top = {bits: orc.gen_primes(10, bits, 1)[0] for bits in DIGITS}
    got = rule([(top[bits], n_in, n_out) for bits, _, n_in, n_out in CASES])
    for (bits, rows, n_in, n_out), (r, tiles, chunks, digits, _) in zip(CASES, got):
        assert (r, digits) == (rows, DIGITS[bits]), (bits, n_in, n_out)
        assert r * (tiles - 1) < n_out <= r * tiles and chunks * 32 >= n_in
    for rows, shapes in SHAPES.items():
        several = [n_out for _, n_out in shapes if n_out > rows]
        assert several and any(n_out % rows for _, n_out in shapes) and any(n_out % rows == 0 or rows == 32 for _, n_out in shapes)


def test_digits_by_the_largest_word(rule):
    """nd signed bytes hold -128 .. 127 times 256^d: words up to 127 (256^nd - 1) / 255."""
    for nd in range(4, 9):
        most = 127 * (256 ** nd - 1) // 255
        assert rule([(most, 16, 9)])[0][3] == nd
        if nd < 8:
            assert rule([(most + 1, 16, 9)])[0][3] == nd + 1


def test_few_outputs_or_inputs_take_no_tile(rule):
    assert rule([(2 ** 54, 15, 500), (2 ** 54, 500, 8), (2 ** 54, 16, 9)])[:2] == [(0, 0, 0, 0, 0)] * 2
    assert rule([(2 ** 54, 16, 9)])[0][0] == 32


def test_laid_out_matrix_fits_its_buffer(rule):
    """The buffer: outputs in whole 256s, inputs in whole 128s, 16 bytes a lane."""
    sizes = [(2 ** 54, n_in, n_out) for n_in in (16, 17, 31, 32, 33, 127, 128, 129, 600, 2048, 65536)
             for n_out in list(range(9, 600)) + [767, 768, 769, 2048, 65535]]
    for (_, n_in, n_out), (rows, tiles, chunks, _, lanes) in zip(sizes, rule(sizes)):
        assert rows in (32, 64, 128, 256) and n_in <= 32 * chunks and n_out <= rows * tiles
        assert lanes * 16 <= (n_out + 255) // 256 * 256 * ((n_in + 127) // 128 * 128)
