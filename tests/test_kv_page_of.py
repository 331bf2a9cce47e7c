"""Where the cache's kernels look a block of 16 positions up in the page table
(CPU): the quotient block / (page_size / 16), over every length that a 32-bit
kv_len can have."""
import random

import pytest

from test_weight_quantization_ttq_b200 import ttq

LAST = 2 ** 27 - 1     # the block of position 2^31 - 1


@pytest.mark.parametrize("d", [1, 2, 3, 4, 5, 7, 8, 9, 100, 1000, 2047, 2048, 2049, 4093, 4095, 4096])
def test_the_page_of_every_length(d):
    """Around the multiples where a quotient turns, 2^24 pages among them (where 64 bits of a product with 2^40 / d
    are full), and at the largest block."""
    rng = random.Random(d)
    turns = [k * d for k in (0, 1, 2, 2 ** 16, 2 ** 24, 2 ** 25, LAST // d)]
    blocks = [t + e for t in turns for e in (-1, 0, 1)] + [LAST, LAST - 1] + [rng.randrange(LAST) for _ in range(2000)]
    blocks += [rng.randrange(LAST // d) * d + e for _ in range(500) for e in (0, d - 1)]
    for n in blocks:
        if 0 <= n <= LAST:
            assert ttq.ttq_testing_kv_page_of(16 * d, n) == n // d, (d, n)


def test_out_of_range():
    for page, block in [(0, 0), (24, 0), (65552, 0), (16, -1), (16, LAST + 1)]:
        assert ttq.ttq_testing_kv_page_of(page, block) == -1
