"""The rule that chooses between the e4m3 products' kernels (csrc/f8_rule.h), compiled for the host."""

import random

import pytest

from tests.f8_rule import SMS, Choice, kernel


def sizes(n, seed, most_rows=1 << 24):
    """Sizes of all kinds within what the entry points take, rows and columns over their logarithms."""
    rng = random.Random(seed)
    for _ in range(n):
        m = min(most_rows - 1, int(2 ** rng.uniform(0, 24)))
        yield m, int(2 ** rng.uniform(0, 20)), 16 * max(1, int(2 ** rng.uniform(0, 12))), rng.random() < 0.5


@pytest.mark.parametrize("m,n,k,gated,want", [
    (1, 4096, 4096, False, "few"), (8, 4096, 4096, False, "few"), (1, 12288, 4096, False, "mid"), (64, 4096, 4096, False, "mid"),
    (16, 4096, 1024, False, "few"), (1024, 256, 1024, False, "mid"), (1024, 4096, 4096, False, "many"), (2048, 12288, 4096, False, "many"),
    (5, 12288, 4096, True, "mid"), (64, 1024, 4096, True, "mid"), (4095, 12288, 4096, True, "many"), (8, 512, 1024, True, "few")])
def test_the_kernel_by_sizes(m, n, k, gated, want):
    """Where the measured times stand clearly apart."""
    assert kernel(m, n, k, gated) == want


def test_few_rows_are_few():
    for m, n, k, gated in sizes(3000, 1):
        c = Choice(m, n, k, gated)
        assert c.kernel != "few" or m <= 32
        assert 128 <= c.wide <= 256 and c.wide % 32 == 0
        assert 16 <= c.rows <= (128 if gated else 256) and c.rows % 16 == 0 and c.split in (1, 2, 4, 8)
        assert c.rows * c.down >= m and 2 * c.split <= max(2, -(-k // 128))
        assert SMS == 152
