"""Differential decode attention (the difference of two softmax maps over one cache) against fp64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from conftest import cuda_available
from eviction_testlib import EPS32, Pool, errors, score_error, softmax64

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]


def make_q(B, Hq, d, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((B, Hq, d)).astype(np.float16)).cuda()


def check(pool, q, lam, gain, eps, scale, out, table=None, x=None):
    q, lam, out = q.cpu().numpy().astype(np.float64), lam.cpu().numpy().astype(np.float64), out.cpu().numpy()
    B, Hq, d = q.shape
    r, half, s = Hq // pool.Hkv, d // 2, (d // 2) ** -0.5
    for b, n in enumerate(pool.lens):
        if n == 0:
            assert not out[b].any()
            continue
        K, V = pool.values(b, n, x)
        for hq in range(Hq):
            k, v = K[hq // r], V[hq // r]
            o, tol = 0.0, 0.0
            for part, f in ((slice(0, half), 1.0), (slice(half, d), -lam[hq])):
                z = q[b, hq, part] @ k[:, part].T * s
                dz = score_error(q[b, hq:hq + 1, part], k[:, part], s)
                o = o + f * (softmax64(z) @ v)
                tol += abs(f) * errors(z, v, dz)[0]
            tol += 2 * EPS32 * np.abs(o).max()
            if gain is not None:
                # a shift of up to tol in every element moves the root mean square by up to tol
                rms, g = np.sqrt((o ** 2).mean() + eps), gain.cpu().numpy().astype(np.float64)
                tol = tol / rms * (1 + np.abs(o) / rms) * np.abs(g) + 12 * EPS32 * np.abs(o / rms * g)
                o = o / rms * g
            err = np.abs(out[b, hq] - o * scale)
            assert (err <= tol * abs(scale) + 2 * EPS32 * np.abs(o * scale)).all(), (b, hq, err.max(), np.max(tol))


@pytest.mark.parametrize("Hkv,r,d,P,Gk,Gv,lens", [
    (8, 1, 128, 16, 64, 128, [513]), (3, 1, 128, 16, 64, 64, [1, 0, 16, 17, 700]), (2, 2, 128, 16, 32, 32, [15, 1024]),
    (2, 4, 128, 16, 64, 128, [2049, 5]), (1, 3, 128, 32, 32, 128, [300, 31]), (2, 4, 128, 64, 64, 64, [63, 65, 999]),
    (4, 1, 64, 16, 32, 64, [255, 1]), (2, 3, 64, 32, 32, 32, [400]), (4, 1, 256, 16, 64, 128, [300, 17]),
    (2, 2, 256, 64, 128, 32, [129, 0, 640]), (1, 1, 256, 16, 128, 64, [5000]),
])
@pytest.mark.parametrize("norm", [False, True])
def test_matches_fp64(kvq, Hkv, r, d, P, Gk, Gv, lens, norm):
    pool = Pool("int4", Hkv, d, lens, P, Gk, Gv, seed=d + r, poison=True)
    q, cfg = make_q(len(lens), Hkv * r, d, 3), pool.cfg(kvq)
    lam = torch.linspace(-0.5, 1.2, Hkv * r, device="cuda")
    gain = torch.randn(d, device="cuda") if norm else None
    out = torch.full((len(lens), Hkv * r, d), float("nan"), device="cuda")
    ws = kvq.new_diff_workspace(cfg, len(lens), Hkv * r, max(lens))
    kvq.kvq_diff_decode_attention(cfg, pool.gpu(), q, pool.table_gpu(), pool.lens_gpu(), max(lens), (d // 2) ** -0.5,
                                  lam, gain, 1e-5, 0.3, out, ws)
    assert kvq.kvq_read_status(ws) == 0
    check(pool, q, lam, gain, 1e-5, 0.3, out)


def test_many_sequences(kvq):
    lens = [(7 * b) % 40 for b in range(300)]
    pool = Pool("int4", 2, 64, lens, 16, 32, 64, seed=9)
    q, cfg = make_q(300, 4, 64, 5), pool.cfg(kvq)
    lam, gain = torch.rand(4, device="cuda"), torch.rand(64, device="cuda")
    out, ws = torch.empty(300, 4, 64, device="cuda"), kvq.new_diff_workspace(cfg, 300, 4, 39)
    kvq.kvq_diff_decode_attention(cfg, pool.gpu(), q, pool.table_gpu(), pool.lens_gpu(), 39, 32 ** -0.5, lam, gain,
                                  1e-6, 1.0, out, ws)
    assert kvq.kvq_read_status(ws) == 0
    check(pool, q, lam, gain, 1e-6, 1.0, out)


def test_thousands_of_short_sequences(kvq):
    lens = [1 + (7 * b) % 40 for b in range(2100)]
    for Hkv in (1, 2):  # one head to a unit, two heads to a unit
        pool = Pool("int4", Hkv, 128, lens, 16, 64, 128, seed=9)
        q, cfg = make_q(2100, Hkv, 128, 5), pool.cfg(kvq)
        lam, out = torch.rand(Hkv, device="cuda"), torch.empty(2100, Hkv, 128, device="cuda")
        ws = kvq.new_diff_workspace(cfg, 2100, Hkv, 40)
        kvq.kvq_diff_decode_attention(cfg, pool.gpu(), q, pool.table_gpu(), pool.lens_gpu(), 40, 0.125, lam, None, 0.0,
                                      1.0, out, ws)
        assert kvq.kvq_read_status(ws) == 0
        check(pool, q, lam, None, 0.0, 1.0, out)


def test_empty_sequence_without_eps_gives_zeros(kvq):
    pool = Pool("int4", 2, 128, [0, 20], 16, 64, 128, seed=9)
    q, cfg = make_q(2, 2, 128, 5), pool.cfg(kvq)
    out, ws = torch.full((2, 2, 128), 7.0, device="cuda"), kvq.new_diff_workspace(cfg, 2, 2, 20)
    kvq.kvq_diff_decode_attention(cfg, pool.gpu(), q, pool.table_gpu(), pool.lens_gpu(), 20, 0.125,
                                  torch.rand(2, device="cuda"), torch.ones(128, device="cuda"), 0.0, 1.0, out, ws)
    assert not out[0].any() and torch.isfinite(out[1]).all()


def test_step_graph_and_stream(kvq):
    from int4_group_quantized_kvq_gb300.cache import PagedKVCache
    for Hkv, r, d, P in ((8, 1, 128, 16), (2, 4, 128, 32), (2, 2, 256, 16)):
        pool = Pool("int4", Hkv, d, [64, 17, 200], P, 64, 64, seed=21)
        x1, q, cfg = pool.gpu(), make_q(3, Hkv * r, d, 8), pool.cfg(kvq)
        x2 = x1.clone()
        k, v = make_q(3, Hkv, d, 30), make_q(3, Hkv, d, 31)
        pos = torch.tensor([63, 16, -1], dtype=torch.int32, device="cuda")
        lam, gain = torch.rand(Hkv * r, device="cuda"), torch.rand(d, device="cuda")
        one = PagedKVCache(cfg, pool.table_gpu(), Hkv * r, 200, pool=x1, diff=True)
        o1, o2 = torch.empty(3, Hkv * r, d, device="cuda"), torch.empty(3, Hkv * r, d, device="cuda")
        lens = pool.lens_gpu()
        one.decode_step_diff(q, k, v, lam, pos, lens, o1, norm_weight=gain)
        for b in (0, 1):
            kvq.kvq_quantize_append(cfg, x2, k[b:b + 1, None].contiguous(), v[b:b + 1, None].contiguous(),
                                    pool.table_gpu()[b:b + 1].contiguous(), pos[b:b + 1].contiguous())
        two = PagedKVCache(cfg, pool.table_gpu(), Hkv * r, 200, pool=x2, diff=True)
        two.attend_diff(q, lam, lens, o2, norm_weight=gain)
        assert one.flags() == 0 and two.flags() == 0
        assert torch.equal(x1, x2) and torch.equal(o1, o2)
        check(pool, q, lam, gain, 1e-5, 1.0, o1, x=x1.cpu().numpy().reshape(pool.bytes.shape))
        o3 = torch.zeros_like(o1)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            two.attend_diff(q, lam, lens, o3, norm_weight=gain)
        graph.replay()
        assert torch.equal(o1, o3)
        side, o4 = torch.cuda.Stream(), torch.zeros_like(o1)
        side.wait_stream(torch.cuda.current_stream())
        two.attend_diff(q, lam, lens, o4, norm_weight=gain, stream=side)
        side.synchronize()
        assert torch.equal(o1, o4)


def test_bad_page_is_flagged(kvq):
    pool = Pool("int4", 2, 128, [100, 50], 16, 64, 128, seed=5)
    q, cfg, table = make_q(2, 4, 128, 9), pool.cfg(kvq), pool.table_gpu()
    table[0, 2] = -9
    ws = kvq.new_diff_workspace(cfg, 2, 4, 100)
    kvq.kvq_diff_decode_attention(cfg, pool.gpu(), q, table, pool.lens_gpu(), 100, 0.1, torch.rand(4, device="cuda"), None,
                                  0.0, 1.0, torch.empty(2, 4, 128, device="cuda"), ws)
    assert kvq.kvq_read_status(ws) == kvq.KVQ_FLAG_BAD_PAGE


def test_tensors_are_checked(kvq):
    pool = Pool("int4", 2, 128, [100, 50], 16, 64, 128, seed=5)
    q, cfg = make_q(2, 4, 128, 9), pool.cfg(kvq)
    lam, gain = torch.rand(4, device="cuda"), torch.rand(128, device="cuda")
    base = dict(cfg=cfg, pool=pool.gpu(), q=q, block_table=pool.table_gpu(), seq_lens=pool.lens_gpu(), max_len=100,
                softmax_scale=0.1, lam=lam, norm_weight=gain, norm_eps=1e-5, out_scale=1.0,
                out=torch.empty(2, 4, 128, device="cuda"), workspace=kvq.new_diff_workspace(cfg, 2, 4, 100))
    kvq.kvq_diff_decode_attention(**base)
    for bad in (dict(lam=lam[:3]), dict(lam=lam.half()), dict(lam=None), dict(norm_weight=gain[:64]),
                dict(norm_weight=gain.cpu()), dict(q=q[:, :, :64].contiguous())):
        with pytest.raises(ValueError):
            kvq.kvq_diff_decode_attention(**{**base, **bad})
    for bad in (dict(norm_eps=-1.0), dict(norm_eps=float("nan")), dict(workspace=base["workspace"][:512].clone())):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_diff_decode_attention(**{**base, **bad})


def test_a_cache_with_a_window_has_no_differential_attention(kvq):
    from int4_group_quantized_kvq_gb300.cache import PagedKVCache
    with pytest.raises(ValueError):
        PagedKVCache(kvq.config(2, 128, 16, 64, 128, 8), torch.arange(8, dtype=torch.int32).view(1, 8), 4, 128,
                     window=16, diff=True)
