"""Parts of an item merged where all scores are large: what counts is how far apart they are."""
from __future__ import annotations

import numpy as np
import pytest

from conftest import cuda_available
from rows_pages_testlib import Kv, Latents

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]

KINDS = {"few": lambda: Kv(64, 4, 64, 32, rows=1), "few 128": lambda: Kv(128, 8, 64, 64, rows=4),
         "many": lambda: Kv(64, 8, 64, 32, rows=20), "many 128": lambda: Kv(128, 4, 64, 64, rows=9),
         "latent": lambda: Latents(256, 16, 64, 64, rows=1), "latent 512": lambda: Latents(512, 64, 64, 64, rows=1)}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [16, 18, 20])
@pytest.mark.parametrize("ahead", [1, 3, 5, -2])
@pytest.mark.parametrize("special", [1, 12])  # (12: several parts start on them)
def test_large_scores_a_little_apart(kvq, kind, size, ahead, special):
    """Scores of 2^size, and 2^size + ahead on `special` pages of 625, whose values are 1 and the others' 0.  Every product
    and sum of a score is exact in fp32 (2^size and small whole numbers and halves), and so is the difference of two
    scores; times log2 e, two roundings, it is off by 2^-21 at most, and a weight by as much.  The weights are rounded
    to fp16 before their product with the values, and the output once: half a step each; fp32 sums: 2^-14 is ample."""
    c = KINDS[kind]()
    n = 40000
    q = np.zeros((c.heads, c.d), np.float16)
    q[:, :32], q[:, c.G] = 2.0 ** (size - 7), 1.0  # 32 dimensions of code 4; one more of the next group
    group = np.arange(c.d) // c.G
    base = np.where(group == 0, 4, 0)
    extra = base.copy()
    extra[c.G] = ahead
    ones = np.ones(c.d // c.G)
    if c.latent:  # the last dimension is the value's mark, which no query looks at
        extra[-1] = 1
        usual, page = (base, ones, np.zeros(64)), (extra, ones, np.zeros(64))
        look = slice(c.d - 1, None)
    else:
        usual, page = c.row((base, 1.0, 0, 1.0)), c.row((extra, 1.0, 1, 1.0))
        look = slice(None)
    table = np.zeros((1, n // c.P), np.int32)
    table[0, 200:200 + special] = 1
    got = c.run(kvq, [[usual] * c.P, [page] * c.P], table, [n], [c.rows], q, 1.0)[:, :, look]
    for i in range(c.rows):
        t = special * c.P * np.exp(float(ahead))
        want = t / (t + n - c.rows + i + 1 - special * c.P)
        assert (np.abs(got[i] - want) <= want * (2 * 2.0 ** -11 + 2.0 ** -14)).all(), (i, float(got[i].min()), float(got[i].max()), want)
