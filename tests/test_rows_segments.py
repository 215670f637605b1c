"""Attention of many rows where a CTA's segments alternate between two row tiles and one, with one tile of positions
and with several: the streams of the kernel hand their outputs over in another way in each."""
from __future__ import annotations

import pytest
import torch

from conftest import cuda_available
from test_rows_attention import Chunk

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("order", [(0, 1), (0, 2), (0, 0, 1, 1), (0, 1, 2), (0, 0, 2, 2, 0, 1), (1, 2, 2, 1, 0)])
def test_two_row_tiles_and_one_in_turn(kvq, d, order):
    # rows, positions: two row tiles of 32 tokens; one row tile and one tile of positions; one row tile and several
    kinds = [(49, 200), (20, 100), (9, 390)]
    n = 240 // len(order)
    new, total = zip(*[kinds[k] for k in order] * n)
    assert sum(new) * 4 > 32 * len(new)
    c = Chunk(kvq, 3, 4, d, 16, 32, 64, list(new), list(total), pad=2, seed=len(order))
    first = c.run().clone()
    c.check(rows=[0, 8, 31, 32, 48])
    for _ in range(20):
        c.out.fill_(7)
        assert torch.equal(c.run(), first)
