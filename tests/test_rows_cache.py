"""The calls on ragged batches of rows run together, as a serving program uses them: through the cache classes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from conftest import cuda_available
from rows_testlib import LatentPool, angles, attend64, ragged, turned

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(got, q, kv, new, total, cu, r, scale):
    for b, (m, n) in enumerate(zip(new, total)):
        for h in range(q.shape[1]):
            K, V = kv(b, h // r, n)
            want, tol = attend64(q[cu[b]:cu[b] + m, h].astype(np.float64), K, V, n - m, scale)
            err = np.abs(got[cu[b]:cu[b] + m, h].astype(np.float64) - want)
            assert (err <= tol).all(), (b, h, float(err.max()))


@pytest.mark.parametrize("rotary", [True, False])
def test_prompt_in_parts_then_decode(kvq, rotary):
    """Two prompts in three uneven parts, then a decode step by the old call: every output against attention over
    what the oracle stores."""
    from int4_group_quantized_kvq_gb300.cache import PagedKVCache
    Hq, Hkv, d, P, B = 8, 2, 128, 16, 2
    cfg, rng = kvq.config(Hkv, d, P, 64, 128, 40), np.random.default_rng(0)
    table = rng.permutation(40)[:2 * 18].reshape(B, 18).astype(np.int32)
    cs = angles(300, d)
    cache = PagedKVCache(cfg, torch.from_numpy(table), Hq, 288, rows=True, rope=kvq.rope(d) if rotary else None,
                         cos_sin=dev(cs) if rotary else None)
    L = oracle.Layout(Hkv, d, P, 64, 128, 40)
    pool = np.zeros(L.pool_bytes, np.uint8)
    done = [0, 0]

    def stored(b, h, n):
        k, v = oracle.dequantize(L, pool, table, b, 0, n)
        return k[:, h].astype(np.float64), v[:, h].astype(np.float64)

    for new in ([130, 7], [1, 100], [60, 0]):
        cu, T = ragged(new)
        q, k, v = (rng.standard_normal((T, H, d)).astype(np.float16) for H in (Hq, Hkv, Hkv))
        gq, out = dev(q), torch.zeros((T, Hq, d), dtype=torch.float16, device="cuda")
        total = [a + n for a, n in zip(done, new)]
        cache.prompt_step(gq, dev(k), dev(v), ints(done), ints(total), ints(cu), out)
        if rotary:
            pos = np.concatenate([a + np.arange(n) for a, n in zip(done, new)])
            q, k = turned(q, cs[pos], d, False), turned(k, cs[pos], d, False)
            assert np.array_equal(gq.cpu().numpy(), q)
        for b, n in enumerate(new):
            if n:
                oracle.quantize_append(L, pool, k[None, cu[b]:cu[b] + n], v[None, cu[b]:cu[b] + n], table[b:b + 1],
                                       np.array([done[b]], np.int32))
        done = total
        assert np.array_equal(cache.pool.cpu().numpy(), pool)
        check(out.cpu().numpy(), q, stored, new, total, cu, Hq // Hkv, cache.softmax_scale)
    rows = ints([0, done[0], done[0] + done[1]])
    ok, ov = (torch.zeros((sum(done), Hkv, d), dtype=torch.float32, device="cuda") for _ in range(2))
    cache.read_rows(ints([0, 0]), rows, ok, ov)
    assert np.array_equal(ok.cpu().numpy()[:done[0]], oracle.dequantize(L, pool, table, 0, 0, done[0])[0])
    # a decode step by kvq_decode_step over the same pool
    q, k, v = (rng.standard_normal((B, H, d)).astype(np.float16) for H in (Hq, Hkv, Hkv))
    out = torch.zeros((B, Hq, d), dtype=torch.float32, device="cuda")
    cache.decode_step(dev(q), dev(k), dev(v), ints(done), ints([n + 1 for n in done]), out)
    for b in range(B):
        oracle.quantize_append(L, pool, k[b:b + 1, None], v[b:b + 1, None], table[b:b + 1], np.array([done[b]], np.int32))
    ref = oracle.decode_attention(L, pool, q, table, np.array([n + 1 for n in done], np.int32), d ** -0.5)
    assert np.abs(out.cpu().numpy() - ref).max() < 2e-4
    assert cache.flags() == 0


def test_latent_prompt_then_decode_captured(kvq):
    """Prompts into a latent cache, then decode steps by a captured graph whose inputs change in place."""
    from int4_group_quantized_kvq_gb300.cache import LatentKVCache
    Lt, R, H, B = 512, 64, 16, 3
    pool = LatentPool(Lt, [260, 90, 130], 64, 64, poison=False)
    cfg, rng, cs = pool.cfg(kvq), np.random.default_rng(1), angles(300, R)
    gain = (1 + 0.1 * rng.standard_normal(Lt)).astype(np.float32)
    cache = LatentKVCache(cfg, torch.from_numpy(pool.table), H, 260, kvq.rope(R), dev(cs), 0.04, dev(gain))
    done = [0, 0, 0]

    def held(b, h, n):
        x = pool.rows(b, n, cache.pool.cpu().numpy())
        return x, x[:, :Lt]

    def rows(T):
        return (rng.standard_normal((T, Lt + R)).astype(np.float16), rng.standard_normal((T, H, R)).astype(np.float16),
                rng.standard_normal((T, H, Lt + R)).astype(np.float16))

    for new in ([255, 80, 1], [1, 3, 120]):
        cu, T = ragged(new)
        x, qpe, q = rows(T)
        gq, out = dev(q), torch.zeros((T, H, Lt), dtype=torch.float16, device="cuda")
        total = [a + n for a, n in zip(done, new)]
        cache.step(dev(x), dev(qpe), gq, ints(done), ints(total), ints(cu), out)
        pos = np.concatenate([a + np.arange(n) for a, n in zip(done, new)])
        q[:, :, Lt:] = turned(qpe, cs[pos], R, False)
        assert np.array_equal(gq.cpu().numpy(), q)
        check(out.cpu().numpy(), q, held, new, total, cu, H, 0.04)
        done = total
    x, qpe, q = rows(B)
    gx, gp, gq, start, lens, cu = dev(x), dev(qpe), dev(q), ints(done), ints([n + 1 for n in done]), ints([0, 1, 2, 3])
    out = torch.zeros((B, H, Lt), dtype=torch.float16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.step(gx, gp, gq, start, lens, cu, out)
    for _ in range(3):
        x, qpe, q = rows(B)
        gx.copy_(dev(x)), gp.copy_(dev(qpe)), gq.copy_(dev(q))
        start.copy_(ints(done)), lens.copy_(ints([n + 1 for n in done]))
        graph.replay()
        torch.cuda.synchronize()
        q[:, :, Lt:] = turned(qpe, cs[np.array(done)], R, False)
        done = [n + 1 for n in done]
        check(out.cpu().numpy(), q, held, [1, 1, 1], done, [0, 1, 2], H, 0.04)
    back = torch.zeros((done[1], Lt + R), dtype=torch.float16, device="cuda")
    cache.read_rows(ints([0, 0, 0]), ints([0, 0, done[1], done[1]]), back)
    assert np.array_equal(back.cpu().numpy(), pool.rows(1, done[1], cache.pool.cpu().numpy()).astype(np.float16))
    assert cache.flags() == 0


def test_cache_refuses(kvq):
    from int4_group_quantized_kvq_gb300.cache import PagedKVCache
    cfg, bt = kvq.config(2, 128, 16, 64, 128, 4), torch.zeros((1, 4), dtype=torch.int32)
    q = torch.zeros((1, 4, 128), dtype=torch.float16, device="cuda")
    one = ints([0, 1])
    with pytest.raises(ValueError):
        PagedKVCache(cfg, bt, 4, 64, rope=kvq.rope(128))
    with pytest.raises(ValueError):
        PagedKVCache(cfg, bt, 4, 64).append_rotary(q, q[:, :2], q[:, :2], q, ints([0]), one)
    with pytest.raises(ValueError):
        PagedKVCache(cfg, bt, 4, 64).attend_rows(q, ints([1]), one, q)
    for k in (dict(window=8), dict(track_weights=True)):
        with pytest.raises(ValueError):
            PagedKVCache(cfg, bt, 4, 64, rows=True, **k)
