"""Refusals of the eviction and differential-attention calls: decided on the host, before the device is touched."""
from __future__ import annotations

import ctypes as C

import pytest


@pytest.fixture(scope="module")
def kvq():
    from int4_group_quantized_kvq_gb300 import _build
    _build.build()
    import int4_group_quantized_kvq_gb300 as pkg
    return pkg


def weights_args(kvq, cfg, **k):
    a = dict(cfg=C.byref(cfg), pool=0x1000, q=0x2000, bt=0x3000, blocks=4, lens=0x4000, B=1, Hq=8, max_len=10,
             scale=1.0, decay=1.0, w=0x5000, stride=10, out=0x6000, ws=0x7000, n=1 << 30, stream=None)
    a.update(k)
    return tuple(a.values())


def test_weights_calls_refuse(kvq):
    L = kvq.lib()
    cfg, cfg64 = kvq.config(8, 128, 16, 64, 128, 10), kvq.config(8, 64, 16, 32, 64, 10)
    for fn in (L.kvq_decode_attention_weights, L.kvq_int8_decode_attention_weights):
        for bad, code in ((dict(w=None), 1), (dict(w=0x5002), 1), (dict(stride=9), 1), (dict(decay=-0.1), 1),
                          (dict(decay=1.01), 1), (dict(decay=float("nan")), 1), (dict(pool=0x1008), 1),
                          (dict(out=None), 1), (dict(ws=0x7010), 1), (dict(Hq=12), 1), (dict(Hq=72), 2),
                          (dict(B=-1), 1), (dict(B=5000), 2), (dict(blocks=0), 1), (dict(max_len=-1), 1),
                          (dict(max_len=(1 << 30) + 1, stride=(1 << 30) + 1), 2), (dict(lens=0x4002), 1)):
            assert fn(*weights_args(kvq, cfg, **bad)) == code, bad
            assert kvq.kvq_last_error()
        assert fn(*weights_args(kvq, cfg, B=0, w=None, pool=None)) == kvq.KVQ_OK
    assert L.kvq_int8_decode_attention_weights(*weights_args(kvq, cfg64)) == kvq.KVQ_EUNSUPPORTED
    big = kvq.config(2, 256, 16, 64, 128, 10)
    assert L.kvq_decode_attention_weights(*weights_args(kvq, big, Hq=10)) == kvq.KVQ_EUNSUPPORTED
    assert L.kvq_decode_step_weights(C.byref(cfg), 0x1000, None, 0x2000, 0x3000, 0x4000, 0x5000, 4, 0x6000, 1, 8, 10,
                                     1.0, 1.0, 0x7000, 10, 0x8000, 0x9000, 1 << 30, None) == kvq.KVQ_EINVAL
    bad = kvq.config(8, 128, 24, 64, 128, 10)
    assert L.kvq_decode_weights_workspace_bytes(C.byref(bad), 1, 8, 10) == 0
    assert L.kvq_decode_weights_workspace_bytes(C.byref(cfg), 1, 12, 10) == 0
    assert L.kvq_int8_decode_weights_workspace_bytes(C.byref(cfg64), 1, 8, 10) == 0


def test_select_refuses(kvq):
    L, cfg = kvq.lib(), kvq.config(8, 128, 16, 64, 128, 10)

    def call(**k):
        a = dict(cfg=C.byref(cfg), w=0x1000, stride=100, lens=0x2000, B=1, max_len=100, keep=10, sinks=2, recent=3,
                 kept=0x3000, new=0x4000, status=None, stream=None)
        a.update(k)
        return L.kvq_evict_select(*a.values())

    for bad, code in ((dict(w=None), 1), (dict(kept=None), 1), (dict(new=None), 1), (dict(lens=None), 1),
                      (dict(stride=99), 1), (dict(keep=0), 1), (dict(keep=4), 1), (dict(sinks=-1), 1),
                      (dict(recent=-1), 1), (dict(recent=0x7fffffff, sinks=0x7fffffff), 1), (dict(B=-1), 1),
                      (dict(new=0x2000), 1), (dict(max_len=(1 << 30) + 1, stride=(1 << 30) + 1), 2),
                      (dict(max_len=-1), 1), (dict(w=0x1001), 1), (dict(status=0x5001), 1), (dict(B=70000), 2)):
        assert call(**bad) == code, bad
        assert kvq.kvq_last_error()
    assert call(B=0, w=None) == kvq.KVQ_OK


def test_compact_refuses(kvq):
    L, cfg = kvq.lib(), kvq.config(8, 128, 16, 64, 128, 10)
    for fn in (L.kvq_evict_compact, L.kvq_int8_evict_compact):
        def call(**k):
            a = dict(cfg=C.byref(cfg), pool=0x1000, bt=0x2000, blocks=4, dst=0x3000, dblocks=4, lens=0x4000, B=1,
                     kept=0x5000, keep=10, w=0x6000, stride=64, status=None, stream=None)
            a.update(k)
            return fn(*a.values())

        for bad, code in ((dict(pool=None), 1), (dict(pool=0x1008), 1), (dict(bt=None), 1), (dict(dst=None), 1),
                          (dict(blocks=0), 1), (dict(dblocks=0), 1), (dict(lens=None), 1), (dict(kept=None), 1),
                          (dict(keep=0), 1), (dict(stride=-1), 1), (dict(w=0x6002), 1), (dict(B=-1), 1),
                          (dict(B=70000), 2)):
            assert call(**bad) == code, bad
            assert kvq.kvq_last_error()
        assert call(B=0, pool=None) == kvq.KVQ_OK


def test_differential_calls_refuse(kvq):
    L = kvq.lib()

    def call(cfg=None, **k):
        cfg = cfg or kvq.config(8, 128, 16, 64, 128, 10)
        a = dict(cfg=C.byref(cfg), pool=0x1000, q=0x2000, bt=0x3000, blocks=4, lens=0x4000, B=1, Hq=8, max_len=10,
                 scale=1.0, lam=0x5000, gain=0x6000, eps=1e-5, out_scale=1.0, out=0x7000, ws=0x8000, n=1 << 30,
                 stream=None)
        a.update(k)
        return L.kvq_diff_decode_attention(*a.values())

    for bad, code in ((dict(lam=None), 1), (dict(lam=0x5002), 1), (dict(gain=0x6004), 1), (dict(eps=-1.0), 1),
                      (dict(eps=float("inf")), 1), (dict(Hq=40), 2), (dict(Hq=12), 1), (dict(q=None), 1),
                      (dict(ws=0x8010), 1), (dict(B=-2), 1)):
        assert call(**bad) == code, bad
        assert kvq.kvq_last_error()
    # a K group across both halves; more query heads than the kernel's slots
    assert call(kvq.config(8, 128, 16, 128, 128, 10)) == kvq.KVQ_EUNSUPPORTED
    assert call(kvq.config(8, 64, 16, 64, 64, 10)) == kvq.KVQ_EUNSUPPORTED
    assert call(kvq.config(2, 256, 16, 64, 128, 10), Hq=6) == kvq.KVQ_EUNSUPPORTED
    assert call(kvq.config(8, 256, 16, 32, 128, 10)) == kvq.KVQ_EUNSUPPORTED
    assert call(B=0, lam=None) == kvq.KVQ_OK
    assert L.kvq_diff_decode_workspace_bytes(C.byref(kvq.config(8, 128, 16, 128, 128, 10)), 1, 8, 10) == 0


def test_binding_refuses_host_tensors(kvq, monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    cfg = kvq.config(2, 128, 16, 64, 128, 4)
    z = torch.zeros(1, 2, 16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        kvq.kvq_evict_select(cfg, z, i, 16, 4, 0, 0, torch.zeros(1, 2, 4, dtype=torch.int32), i)
    with pytest.raises(ValueError):
        kvq.kvq_evict_select(cfg, z, [16], 16, 4, 0, 0, torch.zeros(1, 2, 4, dtype=torch.int32), i)
    with pytest.raises(ValueError):
        kvq.kvq_decode_attention_weights(cfg, torch.zeros(99999, dtype=torch.uint8), torch.zeros(1, 2, 128).half(),
                                         torch.zeros(1, 4, dtype=torch.int32), i, 16, 1.0, 1.0, z,
                                         torch.zeros(1, 2, 128), torch.zeros(9, dtype=torch.uint8))


def test_select_refuses_lengths_that_overlap(kvq):
    L, cfg = kvq.lib(), kvq.config(8, 128, 16, 64, 128, 10)
    for off in (-12, -4, 0, 4, 12):  # of 4 lengths, 16 bytes
        assert L.kvq_evict_select(C.byref(cfg), 0x1000, 100, 0x2000, 4, 100, 10, 2, 3, 0x3000, 0x2000 + off, None,
                                  None) == kvq.KVQ_EINVAL
        assert "overlap" in kvq.kvq_last_error()


def test_select_refuses_budgets_past_its_position_arithmetic(kvq):
    L, cfg = kvq.lib(), kvq.config(8, 128, 16, 64, 128, 10)
    for keep in ((1 << 30) + 1, (1 << 31) - 8192, (1 << 31) - 1):
        assert L.kvq_evict_select(C.byref(cfg), 0x1000, 100, 0x2000, 1, 100, keep, 2, 3, 0x3000, 0x4000, None,
                                  None) == kvq.KVQ_EUNSUPPORTED
        assert "keep" in kvq.kvq_last_error()


def test_weights_wait_test_refuses(kvq):
    L, cfg = kvq.lib(), kvq.config(8, 128, 16, 64, 128, 10)
    args = weights_args(kvq, cfg)
    for limit in (0, 999, 10_000_001):
        assert L.kvq_test_decode_weights_wait_timeout(*args[:-1], limit, None) == kvq.KVQ_EINVAL
        assert "wait_limit_ns" in kvq.kvq_last_error()
    assert L.kvq_test_decode_weights_wait_timeout(*weights_args(kvq, cfg, w=None)[:-1], 1000, None) == kvq.KVQ_EINVAL
