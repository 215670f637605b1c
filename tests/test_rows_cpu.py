"""Refusals of the calls on ragged batches of rows: decided on the host, before the device is touched."""
from __future__ import annotations

import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def kvq():
    from int4_group_quantized_kvq_gb300 import _build
    _build.build()
    import int4_group_quantized_kvq_gb300 as pkg
    return pkg


def caller(fn, **base):
    def call(**k):
        assert set(k) <= set(base)
        return fn(*{**base, **k}.values())
    return call


def sections(kvq, rot, *s):
    return C.byref(kvq.RopeConfig(rot, 0, len(s), (C.c_int32 * 3)(*s)))


def test_rope_append_refuses(kvq):
    cfg, rope = kvq.config(8, 128, 16, 64, 128, 10), kvq.rope(128)
    call = caller(kvq.lib().kvq_rope_append, cfg=C.byref(cfg), rope=C.byref(rope), pool=0x1000, q=0x2000, qs=1024,
                  k=0x3000, ks=1024, v=0x4000, vs=1024, out=0x5000, os=1024, Hq=8, table=0x6000, n=100, pos=None, bt=0x7000,
                  blocks=4, start=0x8000, cu=0x9000, B=1, T=4, status=None, stream=None)
    for bad in (dict(pool=None), dict(pool=0x1008), dict(q=None), dict(q=0x2008), dict(qs=1016), dict(qs=1028),
                dict(k=None), dict(ks=1000), dict(v=0x4002), dict(vs=1 << 40), dict(out=None), dict(out=0x5008), dict(os=8),
                dict(out=0x2000, os=2048), dict(Hq=-1), dict(Hq=1 << 20), dict(table=None), dict(table=0x6004), dict(n=0),
                dict(pos=0x6002), dict(bt=None), dict(bt=0x7001), dict(blocks=0), dict(start=None), dict(cu=None),
                dict(cu=0x9002), dict(B=-1), dict(T=-1), dict(status=0xa001), dict(rope=None), dict(cfg=None),
                dict(T=1 << 27), dict(rope=sections(kvq, 128, 32, 16)), dict(rope=sections(kvq, 128, 32, 32)),
                dict(rope=sections(kvq, 128, 80, -16), pos=0x6000)):
        assert call(**bad) == kvq.KVQ_EINVAL, bad
        assert kvq.kvq_last_error()
    assert call(B=70000) == kvq.KVQ_EUNSUPPORTED
    for rot in (16, 48, 96, 256):
        assert call(rope=C.byref(kvq.rope(rot))) == kvq.KVQ_EUNSUPPORTED
    for inter, axes in ((2, 1), (0, 0), (0, 4)):
        assert call(rope=C.byref(kvq.RopeConfig(128, inter, axes, (C.c_int32 * 3)(64)))) == kvq.KVQ_EINVAL
    assert call(cfg=C.byref(kvq.config(8, 96, 16, 32, 32, 10))) == kvq.KVQ_EUNSUPPORTED
    assert call(B=0, pool=None, k=None) == kvq.KVQ_OK
    assert call(T=0, table=None) == kvq.KVQ_OK


def test_dequantize_varlen_refuses(kvq):
    cfg = kvq.config(8, 128, 16, 64, 128, 10)
    call = caller(kvq.lib().kvq_dequantize_varlen, cfg=C.byref(cfg), pool=0x1000, bt=0x2000, blocks=4, start=0x3000,
                  cu=0x4000, B=1, T=4, k=0x5000, v=0x6000, dtype=0, status=None, stream=None)
    for bad in (dict(pool=None), dict(pool=0x1004), dict(bt=None), dict(blocks=0), dict(start=0x3001), dict(cu=None),
                dict(B=-1), dict(T=-1), dict(k=None), dict(k=0x5008), dict(v=None), dict(v=0x6004), dict(dtype=2),
                dict(status=0x7002)):
        assert call(**bad) == kvq.KVQ_EINVAL, bad
    assert call(T=0, pool=None) == kvq.KVQ_OK


@pytest.mark.parametrize("latent", [False, True])
def test_attention_refuses(kvq, latent):
    cfg = kvq.latent_config(512, 64, 64, 64, 10) if latent else kvq.config(8, 128, 16, 64, 128, 10)
    fn = kvq.lib().kvq_latent_attention if latent else kvq.lib().kvq_chunk_attention
    call = caller(fn, cfg=C.byref(cfg), pool=0x1000, q=0x2000, bt=0x3000, blocks=4, lens=0x4000, cu=0x5000, B=1, T=4, H=16,
                  max_len=64, scale=0.1, out=0x6000, ws=0x7000, n=1 << 40, stream=None)
    for bad in (dict(pool=None), dict(pool=0x1001), dict(q=None), dict(q=0x2008), dict(bt=None), dict(blocks=0),
                dict(lens=None), dict(lens=0x4002), dict(cu=None), dict(B=-1), dict(T=-1), dict(H=0), dict(max_len=-1),
                dict(max_len=(1 << 30) + 1), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None),
                dict(out=0x6004), dict(ws=None), dict(ws=0x7080), dict(T=1 << 28), dict(cfg=None)):
        assert call(**bad) == kvq.KVQ_EINVAL, bad
        assert kvq.kvq_last_error()
    assert call(B=70000) == kvq.KVQ_EUNSUPPORTED
    for scale in (2.1e19, -3e38):
        assert call(scale=scale) == kvq.KVQ_EINVAL
    assert call(T=0, pool=None, ws=None) == kvq.KVQ_OK
    if latent:
        assert call(H=1025) == kvq.KVQ_EINVAL
        for c in ((128, 64, 64, 64, 1), (512, 32, 64, 64, 1), (512, 64, 8, 64, 1), (512, 64, 64, 16, 1)):
            assert call(cfg=C.byref(kvq.latent_config(*c))) == kvq.KVQ_EUNSUPPORTED
        assert call(cfg=C.byref(kvq.latent_config(512, 64, 64, 64, 0))) == kvq.KVQ_EINVAL
    else:
        assert call(H=12) == kvq.KVQ_EINVAL
        assert call(H=72) == kvq.KVQ_EUNSUPPORTED
        assert call(cfg=C.byref(kvq.config(8, 256, 16, 64, 128, 10))) == kvq.KVQ_EUNSUPPORTED


def test_latent_rows_refuse(kvq):
    cfg, rope = kvq.latent_config(512, 64, 64, 64, 10), kvq.rope(64)
    call = caller(kvq.lib().kvq_latent_append, cfg=C.byref(cfg), rope=C.byref(rope), pool=0x1000, x=0x2000, xs=576,
                  gain=0x3000, eps=1e-6, qpe=0x4000, qs=1024, out=0x5000, H=16, table=0x6000, n=100, pos=None, bt=0x7000,
                  blocks=4, start=0x8000, cu=0x9000, B=1, T=4, status=None, stream=None)
    for bad in (dict(pool=None), dict(x=None), dict(x=0x2002), dict(xs=568), dict(xs=580), dict(gain=0x3004),
                dict(eps=-1.0), dict(eps=float("nan")), dict(qpe=None), dict(qs=1016), dict(out=None), dict(out=0x5002),
                dict(H=-1), dict(H=1025), dict(table=None), dict(n=0), dict(bt=None), dict(blocks=0), dict(cu=None), dict(B=-1),
                dict(T=-1), dict(status=0xa001)):
        assert call(**bad) == kvq.KVQ_EINVAL, bad
    assert call(rope=C.byref(kvq.rope(32))) == kvq.KVQ_EUNSUPPORTED
    assert call(rope=sections(kvq, 64, 16, 16), pos=0x6000) == kvq.KVQ_EUNSUPPORTED
    back = caller(kvq.lib().kvq_latent_dequantize, cfg=C.byref(cfg), pool=0x1000, bt=0x2000, blocks=4, start=0x3000, cu=0x4000,
                  B=1, T=4, out=0x5000, status=None, stream=None)
    for bad in (dict(pool=None), dict(out=None), dict(out=0x5008), dict(bt=None), dict(start=None), dict(T=-1)):
        assert back(**bad) == kvq.KVQ_EINVAL, bad


def test_sizes(kvq):
    for L, P, G in ((512, 64, 64), (256, 16, 32), (512, 32, 128)):
        cfg = kvq.latent_config(L, 64, P, G, 7)
        assert kvq.kvq_latent_block_bytes(cfg) == P * (L // 2 + 2 * (L // G) + 128)
        assert kvq.kvq_latent_pool_bytes(cfg) == 7 * kvq.kvq_latent_block_bytes(cfg)
    with pytest.raises(kvq.KvqError):
        kvq.kvq_latent_pool_bytes(kvq.latent_config(300))
    L = kvq.lib()
    cfg = kvq.config(8, 128, 16, 64, 128, 10)
    for bad in ((12, 64), (72, 64), (8, -1)):
        assert L.kvq_chunk_workspace_bytes(C.byref(cfg), 1, *bad) == 0
    assert L.kvq_chunk_workspace_bytes(C.byref(cfg), 0, 8, 64) == 0
    assert L.kvq_latent_workspace_bytes(C.byref(kvq.latent_config(512)), 1, 0, 64) == 0


def test_rope_table(kvq):
    t = kvq.rope_table(1 << 17, 128, device="cpu")
    assert t.dtype == torch.float32 and t.shape == (1 << 17, 128)
    a = (1 << 17) - 1
    want = torch.tensor(float(a), dtype=torch.float64)
    assert t[a, 0] == want.cos().float() and t[a, 64] == want.sin().float()
    f = torch.linspace(0.1, 1, 16, dtype=torch.float64)
    assert torch.equal(kvq.rope_table(5, 32, inv_freq=f, device="cpu")[3, :16], (3 * f).cos().float())
    with pytest.raises(ValueError):
        kvq.rope_table(5, 32, inv_freq=f[:8], device="cpu")
    with pytest.raises(ValueError):
        kvq.rope(64, sections=[8, 8, 8, 8])
    assert list(kvq.rope(64, sections=[16, 8, 8]).sections) == [16, 8, 8]
