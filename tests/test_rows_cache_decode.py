"""Decode steps of a cache with rotary positions: keys of prompts and of decoded tokens are turned alike, whichever calls
bring them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from conftest import cuda_available
from rows_testlib import angles, ragged, turned


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")
@pytest.mark.parametrize("inter", [False, True])
def test_decode_behind_a_rotary_prompt(kvq, inter):
    """A prompt by prompt_step, then decode steps over raw projections (append_rotary, then attend) and over turned ones
    (decode_step), in turn: the pool holds turned keys alone, and the outputs are the oracle's over them."""
    from int4_group_quantized_kvq_gb300.cache import PagedKVCache
    Hq, Hkv, d, P, B, rot = 8, 2, 128, 16, 2, 64
    cfg, rng = kvq.config(Hkv, d, P, 64, 128, 40), np.random.default_rng(2)
    table = rng.permutation(40)[:2 * 18].reshape(B, 18).astype(np.int32)
    cs = angles(300, rot)
    cache = PagedKVCache(cfg, torch.from_numpy(table), Hq, 288, rows=True, rope=kvq.rope(rot, inter), cos_sin=dev(cs))
    L = oracle.Layout(Hkv, d, P, 64, 128, 40)
    pool = np.zeros(L.pool_bytes, np.uint8)
    new = [70, 33]
    cu, T = ragged(new)
    q, k, v = (rng.standard_normal((T, H, d)).astype(np.float16) for H in (Hq, Hkv, Hkv))
    cache.prompt_step(dev(q), dev(k), dev(v), ints([0, 0]), ints(new), ints(cu), torch.zeros((T, Hq, d), dtype=torch.float16,
                                                                                             device="cuda"))
    pos = np.concatenate([np.arange(n) for n in new])
    k = turned(k, cs[pos], rot, inter)
    for b, n in enumerate(new):
        oracle.quantize_append(L, pool, k[None, cu[b]:cu[b] + n], v[None, cu[b]:cu[b] + n], table[b:b + 1],
                               np.array([0], np.int32))
    done = new
    for step in range(4):
        q, k, v = (rng.standard_normal((B, H, d)).astype(np.float16) for H in (Hq, Hkv, Hkv))
        tq, tk = (turned(x, cs[np.array(done)], rot, inter) for x in (q, k))
        lens, out = [n + 1 for n in done], torch.zeros((B, Hq, d), dtype=torch.float32, device="cuda")
        if step % 2 == 0:
            gq = dev(q)
            cache.append_rotary(gq, dev(k), dev(v), gq, ints(done), ints([0, 1, 2]))
            cache.attend(gq, ints(lens), out)
            assert np.array_equal(gq.cpu().numpy(), tq)
        else:
            cache.decode_step(dev(tq), dev(tk), dev(v), ints(done), ints(lens), out)
        for b in range(B):
            oracle.quantize_append(L, pool, tk[b:b + 1, None], v[b:b + 1, None], table[b:b + 1], np.array([done[b]], np.int32))
        assert np.array_equal(cache.pool.cpu().numpy(), pool)
        ref = oracle.decode_attention(L, pool, tq, table, np.array(lens, np.int32), d ** -0.5)
        assert np.abs(out.cpu().numpy() - ref).max() < 2e-4
        done = lens
    assert cache.flags() == 0


def test_the_calls_that_turn_nothing_say_so():
    from int4_group_quantized_kvq_gb300.cache import PagedKVCache
    for call in (PagedKVCache.append, PagedKVCache.decode_step, PagedKVCache.decode_step_diff, PagedKVCache.decode_step_host):
        assert "as it is given" in call.__doc__ or "as they are given" in call.__doc__, call.__name__
