"""Attention over keys and values of very different sizes beside each other: by blocks of tokens, by single tokens, by groups of
64 columns, and in tokens that a row does not see. Every column's bound is that of tests/test_gpu_attn.py, which goes by
what the row itself sees of that column: 2^-8 |out| + 2^-9 (1 + scale sum|q k|) sum p (|v| + 8 s)."""

import numpy as np
import pytest
import torch

from bit_group_quantized_gb300 import lib
from oracle import attn_oracle as A
from oracle import bgq_oracle as O
from tests.test_gpu_attn import Case, attn_close, bf16

pytestmark = pytest.mark.gpu

VALUES, KEYS = 3, 1  # the pairs' places among a case's arrays


def times(c, which, tokens, factor, group=slice(None), b=0):
    """Multiplies the pairs (scale and bias) of these tokens of sequence b by a power of two."""
    for t in tokens:
        at = A.slot(t, b, c.pages, c.page, c.n_pages)
        if at is not None:
            c.np[which][at[0], :, at[1], group] = O.f64_to_bf16_bits(O.bf16_to_f64(c.np[which][at[0], :, at[1], group]) * factor)


def run(c, hq, scale=1.5, **kw):
    q = bf16(c.rng, c.rows, hq, c.d, dev=c.dev, scale=scale)
    out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, want_lse=True, **kw)
    return q, out, lse


ROWS = [1, 4, 64]  # the few-row kernel with one and several rows, the many-row kernel


@pytest.mark.parametrize("new", ROWS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("size", [2.0 ** -8, 2.0 ** -11, 2.0 ** -15, 2.0 ** -30, 2.0 ** 8, 2.0 ** 13])
def test_blocks_of_values_around_a_size(cuda_device, size, d, new):
    """Blocks of 32 tokens by turns a little above and a little below a size at which half precision's range may end."""
    c = Case(cuda_device, [700], [new], 1, d, 16, seed=50)
    for t in range(700):
        times(c, VALUES, [t], size * (2.0 if t // 32 % 2 else 0.125))
    q, out, lse = run(c, 4)
    attn_close(c, q, out, lse)


@pytest.mark.parametrize("new", ROWS)
@pytest.mark.parametrize("before", ["absent", "zeros", "normal", "large"])
@pytest.mark.parametrize("size", [2.0 ** -10, 2.0 ** -16, 2.0 ** -40])
def test_small_values_behind_others(cuda_device, size, before, new):
    """Small values behind a given-up page, a block of zeros, one of ordinary values, one of large ones that a window hides."""
    c = Case(cuda_device, [600], [new], 1, 128, 32, seed=51)
    times(c, VALUES, range(32, 600), size)
    if before == "absent":
        c.pages[0, 0] = -1
    times(c, VALUES, range(32), {"zeros": 0.0, "large": 2.0 ** 60}.get(before, 1.0))
    for window in (0, 500):
        q, out, lse = run(c, 4, window=window)
        attn_close(c, q, out, lse, window=window)


@pytest.mark.parametrize("new", ROWS)
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("factor", [2.0 ** -12, 2.0 ** -20, 2.0 ** -28, 2.0 ** -60, 2.0 ** 20, 2.0 ** 60])
def test_groups_of_values_of_different_sizes(cuda_device, factor, d, new):
    """A group of 64 columns far smaller or larger than the others, in every token, in every other one, in the first half."""
    for tokens in (range(300), range(0, 300, 2), range(150)):
        c = Case(cuda_device, [300], [new], 2, d, 16, seed=52)
        times(c, VALUES, tokens, factor, group=1)
        q, out, lse = run(c, 8)
        attn_close(c, q, out, lse)


@pytest.mark.parametrize("new", ROWS[1:])
@pytest.mark.parametrize("which", [KEYS, VALUES])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("factor", [2.0 ** 24, 2.0 ** 60, 2.0 ** 110])
def test_large_tokens_that_a_row_does_not_see(cuda_device, factor, d, which, new):
    """Finite tokens of any size hidden by causality (the last) and by the window (the first ones) leave the other rows right."""
    c = Case(cuda_device, [300], [new], 1, d, 16, seed=53)
    times(c, which, [299], factor)
    times(c, which, range(0, 300 - new - 100), factor)
    q, out, lse = run(c, 4, window=101)
    o, l, a, s = c.oracle(q, window=101)
    see = slice(0, new - 1)  # all but the last row, which does see a large token
    got = O.bf16_to_f64(out.cpu().view(torch.int16).numpy().astype(np.uint16))
    assert (np.abs(got - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -9 * (1 + s)[..., None] * a)[see].all()
    assert (np.abs(lse.cpu().double().numpy() - l) <= 2.0 ** -10 * (s + 1))[see].all()


@pytest.mark.parametrize("new", ROWS)
@pytest.mark.parametrize("exps", [(0, -9), (0, -25), (20, 0), (3, 40), (-30, -70)])
def test_tokens_of_different_sizes(cuda_device, exps, new):
    """Values by single tokens of two sizes, mixed; then keys."""
    pick = np.random.default_rng(5).random(300) < 0.3
    for which in (VALUES, KEYS):
        c = Case(cuda_device, [300], [new], 1, 128, 16, seed=54)
        for t in range(300):
            times(c, which, [t], 2.0 ** exps[int(pick[t])])
        # large keys: their scores stay within some tens
        q, out, lse = run(c, 4, scale=1.5 if which == VALUES else 1.5 * 2.0 ** -max(exps))
        attn_close(c, q, out, lse)


@pytest.mark.parametrize("new", ROWS)
@pytest.mark.parametrize("high", [6.0, 12.0, 16.0, 18.0])
def test_a_flat_tail_behind_a_high_first_token(cuda_device, high, new):
    """A first token that takes nearly all of the softmax and has a value of zeros: what a row gets is its tail's, thousands of
    tokens whose probabilities are e^-high of the first one's."""
    c = Case(cuda_device, [4000], [new], 1, 128, 16, seed=55)
    for t in range(4000):
        p, at = A.slot(t, 0, c.pages, 16, c.n_pages)
        pair = O.bf16_to_f64(c.np[KEYS][p, :, at]) * 0.02
        c.np[KEYS][p, :, at] = O.f64_to_bf16_bits(pair if t else pair * 0 + [0.0, high / (128 ** 0.5 * 0.8 * 1.5)])
    times(c, VALUES, [0], 0.0)
    q = bf16(c.rng, c.rows, 4, 128, dev=cuda_device, scale=1.5).abs()
    out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, want_lse=True)
    attn_close(c, q, out, lse)


@pytest.mark.parametrize("d,hq,new", [(64, 4, 1), (64, 5, 3), (128, 8, 1), (128, 3, 2)])
@pytest.mark.parametrize("what", ["tokens", "groups", "hidden", "scores"])
def test_many_sequences_of_values_of_different_sizes(cuda_device, what, d, hq, new):
    """More units than SMs, where two blocks share one and have half the registers: the same sizes beside each other.
    Very large scores: the few-row kernel multiplies 64 + code, so that a group's partial sums reach s (64 |sum q| + 15 sum |q|). With
    normal queries |sum q| of 64 stays below 28 (3.5 sigma of 8) and sum |q| near 51, so they reach 2560 s; sum |q k| is near
    51 * 2.4 s (codes of a normal group are 2.4 from its middle on average): 21 times as much. Each of the d/16 + 8 <= 16 partial
    sums and products is off by 2^-23 of itself (accumulation truncates): 16 * 21 * 2^-23 < 2^-14 of scale sum|q k| in all."""
    B = 170
    kv = [3 + 37 * b % 190 for b in range(B)]
    c = Case(cuda_device, kv, [min(new, n) for n in kv], 1, d, 16, seed=56, room=0)
    rng = np.random.default_rng(57)
    P = O.bf16_to_f64(c.np[VALUES])
    window = 0
    if what == "tokens":
        P = P * 2.0 ** np.round(rng.uniform(-40, 40, P.shape[:3] + (1, 1)))
    elif what == "groups":
        P = P * 2.0 ** np.round(rng.uniform(-40, 40, (1, 1, 1, P.shape[3], 1))) * (rng.random(P.shape[:3] + (1, 1)) > 0.2)
    c.np[VALUES] = O.f64_to_bf16_bits(P)
    if what == "hidden":
        window = 30
        for b, n in enumerate(kv):
            times(c, VALUES, range(0, n - window - new, 2), 2.0 ** 70, b=b)
            times(c, KEYS, range(1, n - window - new, 2), 2.0 ** 90, b=b)
    q = bf16(c.rng, c.rows, hq, d, dev=cuda_device, scale=1.5)
    scale = 1e7 * d ** -0.5 if what == "scores" else None
    out, lse = lib.bgq_kv4_attention(c.cache(), c.seqs(), q, scale=scale, window=window, want_lse=True)
    if what != "scores":
        attn_close(c, q, out, lse, window=window)
        return
    o, l, a, s = c.oracle(q, scale=scale)
    gl = lse.cpu().double().numpy()
    assert np.isfinite(out.float().cpu().numpy()).all() and (np.abs(gl - l) <= 2.0 ** -14 * s + np.log(200)).all()
