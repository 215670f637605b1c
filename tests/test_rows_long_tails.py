"""Attention where one position outweighs each of very many others, which together still count."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from conftest import cuda_available
from rows_pages_testlib import Kv, Latents

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]

KINDS = {"few": lambda: Kv(64, 4, 64, 32, rows=1), "few 128": lambda: Kv(128, 8, 64, 64, rows=4),
         "many": lambda: Kv(64, 8, 64, 32, rows=20), "many 128": lambda: Kv(128, 4, 64, 64, rows=40),
         "latent": lambda: Latents(256, 16, 64, 64, rows=1), "latent 512": lambda: Latents(512, 64, 64, 64, rows=1)}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ahead", [10.0, 14.0, 18.0])
def test_the_many_are_not_lost(kvq, kind, ahead):
    """Position 0's score is `ahead` above the 2^17 others', whose value is 1 where its own is 0: the output is
    t / (1 + t), t = (number of the others) e^-ahead.  As many sequences as SMs, so that a sequence is one run of work.

    The largest weight is held in fp16 as 2^7 at least, so that another is off by half a step, 2^-11 of it, or by
    2^-25 / 2^7 of the largest where it is subnormal: 2^17 times that, 2^-15, at most.  The tensor cores add 16
    positions at a time to the output and cut off less than a step of the sum, 2^-23 of it: 2^13 times, 2^-10.  The
    output is rounded to fp16 (2^-11 of it); the sum that divides adds a tile at a time, rounded: 2^-14 for all of it."""
    c = KINDS[kind]()
    n, sms = 1 << 17, torch.cuda.get_device_properties(0).multi_processor_count
    q = np.zeros((c.heads, c.d), np.float16)
    q[:, :c.G] = 1
    if c.latent:
        group, ones, none = np.arange(c.d) // c.G, np.ones(c.d // c.G), np.zeros(64)
        first, other = (np.where(group == 0, 4, 0), ones, none), (np.where(group == 0, 0, 1), ones, none)
        look = slice(c.G, None)
    else:
        first, other = c.row((4, 1.0, 0, 1.0)), c.row((0, 1.0, 1, 1.0))
        look = slice(None)
    pages = [[first] + [other] * (c.P - 1), [other] * c.P]
    table = np.ones((sms, n // c.P), np.int32)
    table[:, 0] = 0
    got = c.run(kvq, pages, table, [n] * sms, [c.rows] * sms, q, ahead / (4 * c.G))[:, :, look]
    for i in (0, c.rows - 1):
        t = (n - c.rows + i) * np.exp(-ahead)
        want, g = t / (1 + t), got[i::c.rows]
        tol = want * (2 * 2.0 ** -11 + 2.0 ** -10 + 2.0 ** -14) + 2.0 ** -15
        assert (np.abs(g - want) <= tol).all(), (i, float(g.min()), float(g.max()), want)
