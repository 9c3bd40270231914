"""Products of ckks_matmul_i8 that reach every tile, whole and ragged, for every
number of digits.  What the library's rule makes of them is checked on the CPU,
their words on the GPU."""

# bits of the primes: signed bytes of a word
DIGITS = {30: 4, 36: 5, 45: 6, 54: 7, 60: 8}

# outputs of a tile: (inputs, outputs), one tile whole or ragged, then several
SHAPES = {32: [(33, 20), (70, 90)], 64: [(70, 64), (140, 190)], 128: [(40, 100), (300, 384)],
          256: [(160, 250), (129, 512), (300, 500)]}

CASES = [(bits, rows, n_in, n_out) for bits in DIGITS for rows, shapes in SHAPES.items() for n_in, n_out in shapes]


def edges(rows, n_out):
    """The outputs on either side of a tile's, a wave's and a register group's borders."""
    at = {0, 3, 4, 31, 32, rows // 2 - 1, rows // 2, rows - 1, rows, n_out - 1}
    return sorted(j for j in at if j < n_out)
