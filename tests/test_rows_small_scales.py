"""Attention over rows whose scales are subnormal or nearly: what is cached is small, not lost.

An element is code x scale, held as half of it in fp16: rounded by at most half a step (2^-11 relative), 2^-25 on the half
where that is subnormal, so 2^-24 on the element."""
from __future__ import annotations

import numpy as np
import pytest

from conftest import cuda_available
from rows_pages_testlib import Kv, Latents

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]

U = 2.0 ** -24
SCALES = [1, 2, 3, 5, 7, 11, 17, 33, 101, 1023, 1025, 1537, 2047, 2048]  # in units of 2^-24
KINDS = {  # few lines to a sequence, many of them in one row tile and in two, and the latent kernel's two widths
    "few": lambda: Kv(64, 1, 64, 32, rows=1), "few 128": lambda: Kv(128, 8, 16, 128, rows=3),
    "many": lambda: Kv(64, 8, 32, 64, rows=7), "many 128": lambda: Kv(128, 4, 16, 64, rows=40),
    "latent": lambda: Latents(256, 5, 32, 64, rows=2), "latent 512": lambda: Latents(512, 16, 64, 128, rows=1),
}


@pytest.mark.parametrize("kind", KINDS)
def test_values(kvq, kind):
    """All positions of a sequence hold the same row: every output is that row (the weights add up to 1, up to their
    rounding and the output's, half a step each)."""
    c, rng = KINDS[kind](), np.random.default_rng(0)
    codes = rng.integers(-7, 8, c.d)
    pages, n = [], c.rows + 2
    for s in SCALES:
        s = np.float16(s * U)
        row = (codes, np.full(c.d // c.G, s), np.zeros(64)) if c.latent else c.row((1, 1.0, codes, s))
        pages.append([row] * c.P)
    table = np.arange(len(pages))[np.arange(len(pages) * -(-n // c.P)) // -(-n // c.P)].reshape(len(pages), -1)
    q = rng.standard_normal((c.heads, c.d)).astype(np.float16)
    got = c.run(kvq, pages, table, [n] * len(pages), [c.rows] * len(pages), q, 0.1)
    for i, s in enumerate(SCALES):
        want = codes * (s * U)
        err = np.abs(got[i * c.rows:(i + 1) * c.rows] - want)
        tol = np.maximum(2.0 ** -11 * np.abs(want), U) + 2 * 2.0 ** -11 * np.abs(want) + U / 2
        assert (err <= 1.01 * tol).all(), (s, float(err.max() / U), float(tol[err.max(axis=(0, 1)).argmax()] / U))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("s", SCALES)
def test_keys(kvq, kind, s):
    """Position 0's key has codes of 6 (half of an element is 3 scales: exact), the others' are 0; the scale of the
    softmax makes its score 2.  Its value is 1, the others' 0, so the output is its weight: rounded, divided by the
    sum of the unrounded ones and rounded again, half a step each."""
    c = KINDS[kind]()
    q = np.zeros((c.heads, c.d), np.float16)
    q[:, :c.G] = 1
    scales = np.ones(c.d // c.G)
    scales[0] = s * U
    if c.latent:
        group = np.arange(c.d) // c.G
        first, other = (np.where(group == 0, 6, 1), scales, np.zeros(64)), (0 * group, scales, np.zeros(64))
        look = slice(c.G, None)
    else:
        first, other = c.row((6, scales, 1, 1.0)), c.row((0, 1.0, 0, 1.0))
        look = slice(None)
    n = c.rows + 1
    pages = [[first] + [other] * (c.P - 1), [other] * c.P]
    table = [[0] + [1] * ((n - 1) // c.P)]
    got = c.run(kvq, pages, table, [n], [c.rows], q, 2.0 / (6 * s * U * c.G))
    for i in range(c.rows):
        want = np.exp(2.0) / (np.exp(2.0) + n - c.rows + i)
        assert (np.abs(got[i, :, look] - want) <= want * (3.1 * 2.0 ** -11)).all(), (i, float(got[i, 0, -1]), want)
