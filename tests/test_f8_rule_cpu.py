"""The rule that chooses between the e4m3 products' kernels (csrc/f8_rule.h), compiled for the host."""

import os
import random
import re

import pytest

from tests.f8_rule import ROOT, SMS, Choice, kernel


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


def test_every_size_has_a_kernel_that_can_launch():
    """A grid's y ends at 65535 and a launch has fewer than 2^31 CTAs; the sizes are all that the entry points take, up to the most
    rows, those among them whose results no memory holds."""
    most = (1 << 24) - 1
    ends = [(m, n, k, g) for m in (16776960, 16776961, most, 65535 * 128, 65535 * 128 + 1) for n in (1, 16, 128, 129, 1 << 20)
            for k in (16, 128, 1024, 65536) for g in (False, True)]
    for m, n, k, gated in ends + list(sizes(3000, 2)):
        for sms in (SMS, 148, 132, 80):
            c = Choice(m, n, k, gated, sms)
            assert min(c.few_us, c.mid_us, c.many_us) > 0
            if c.kernel == "mid":
                assert 1 <= c.down <= 65535 and -(-n // 128) * c.split * c.down < 1 << 31, (m, n, k, gated)
    # 65536 tiles of 256 rows
    assert kernel(16776961, 128, 128) == "many" and kernel(16776960, 128, 128) == "mid"


def test_no_tile_without_rows():
    """Tiles of x's rows as many as hold some; the tiles' rows are rounded up to 16 after x is cut."""
    for m, n, k, gated in [(1078, 128, 4096, False), (1063, 128, 4096, True), (864, 512, 1024, False)]:
        c = Choice(m, n, k, gated)
        assert c.kernel == "mid" and (c.down - 1) * c.rows < m <= c.down * c.rows
    for gated in (False, True):
        for n, k in ((128, 128), (128, 4096), (512, 1024), (1040, 2064), (4096, 4096)):
            for m in range(1, 2100):
                c = Choice(m, n, k, gated)
                assert (c.down - 1) * c.rows < m <= c.down * c.rows, (m, n, k, gated)


def test_smoke_takes_each_kernel():
    """The feed-forward block of the smoke test, 640 wide and 1040 inside, by all three kernels."""
    text = open(os.path.join(ROOT, "__graft_entry__.py"), encoding="utf-8").read()
    rows = [int(m) for m in re.search(r"for m in \(([\d, ]+)\):\n        h = torch.randn\(m, 640", text).group(1).split(",")]
    assert "((1040, 640), (1040, 640), (640, 1040))" in text
    assert [kernel(m, 1040, 640, True) for m in rows] == ["few", "mid", "many"]
    assert [kernel(m, 640, 1040) for m in rows] == ["few", "mid", "many"]
