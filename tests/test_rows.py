"""Rotary append and read-back of ragged batches, and the latent cache's rows: stored bytes and values against numpy."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from conftest import cuda_available
from rows_testlib import angles, ragged, turned

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]


def dev(x, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda() if dtype is None else torch.tensor(x, dtype=dtype, device="cuda")


class Batch:
    """A ragged batch of q, k, v rows in one projection's rows, and a cache for it."""

    def __init__(self, Hq, Hkv, d, P, Gk, Gv, new, start, pad=0, seed=0, scale=1.0):
        rng = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.d, self.P, self.Gk, self.Gv, self.new, self.start = Hq, Hkv, d, P, Gk, Gv, new, start
        self.cu, self.T = ragged(new, pad)
        x = (scale * rng.standard_normal((self.T, (Hq + 2 * Hkv) * d + 8))).astype(np.float16)
        if self.T > 3:  # a row of zeros, large and tiny rows
            x[1], x[2] = 0, (x[2].astype(np.float32) * 2.0 ** -14).astype(np.float16)
            x[3] = (np.sign(x[3]) * 40000).astype(np.float16)
        self.x = x
        pages = [(s + n + P - 1) // P for s, n in zip(start, new)]
        self.blocks, self.num_pages = max(1, max(pages)), sum(pages) + 2
        order = rng.permutation(self.num_pages).astype(np.int32)
        self.table = np.full((len(new), self.blocks), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.seq = np.repeat(np.arange(len(new)), new)
        self.pos = np.asarray(start)[self.seq] + np.arange(self.cu[-1]) - self.cu[self.seq] if len(self.seq) else \
            np.zeros(0, int)

    def parts(self, x):
        q, k, v = (x[:, a * self.d:b * self.d] for a, b in ((0, self.Hq), (self.Hq, self.Hq + self.Hkv),
                                                             (self.Hq + self.Hkv, self.Hq + 2 * self.Hkv)))
        if isinstance(x, torch.Tensor):
            return [t.unflatten(1, (-1, self.d)) for t in (q, k, v)]
        return [t.reshape(len(x), -1, self.d) for t in (q, k, v)]

    def cfg(self, kvq):
        return kvq.config(self.Hkv, self.d, self.P, self.Gk, self.Gv, self.num_pages)

    def places(self):
        return dev(self.table), dev(self.start, torch.int32), dev(self.cu)

    def want_pool(self, k, v):
        L = oracle.Layout(self.Hkv, self.d, self.P, self.Gk, self.Gv, self.num_pages)
        pool = np.full(L.pool_bytes, 0xA5, np.uint8)
        for b, n in enumerate(self.new):
            lo = self.cu[b]
            if n:
                oracle.quantize_append(L, pool, k[None, lo:lo + n], v[None, lo:lo + n], self.table[b:b + 1],
                                       np.array([self.start[b]], np.int32))
        return pool


SHAPES = [  # Hq, Hkv, d, P, Gk, Gv, rot, inter
    (4, 2, 128, 16, 64, 128, 128, False), (3, 3, 128, 32, 32, 32, 64, True), (8, 1, 128, 64, 128, 64, 32, False),
    (2, 2, 64, 16, 32, 64, 64, False), (5, 1, 64, 16, 64, 32, 32, True), (2, 2, 256, 16, 64, 128, 256, False),
    (6, 3, 256, 32, 32, 128, 128, False), (1, 1, 256, 64, 128, 32, 64, True), (7, 7, 128, 16, 64, 64, 64, False),
    (2, 1, 64, 32, 32, 32, 32, False),
]


@pytest.mark.parametrize("Hq,Hkv,d,P,Gk,Gv,rot,inter", SHAPES)
@pytest.mark.parametrize("new,start,pad", [([1], [0], 0), ([5, 0, 17, 1], [3, 9, 0, 15], 3), ([300, 1], [16, 700], 0)])
def test_rope_append(kvq, Hq, Hkv, d, P, Gk, Gv, rot, inter, new, start, pad):
    c = Batch(Hq, Hkv, d, P, Gk, Gv, new, start, pad, seed=d + rot)
    cs = angles(max(s + n for s, n in zip(start, new)), rot)
    q, k, v = c.parts(c.x)
    n = c.cu[-1]
    qt, kt = turned(q[:n], cs[c.pos], rot, inter), turned(k[:n], cs[c.pos], rot, inter)
    x, pool = dev(c.x), torch.full((kvq.kvq_pool_bytes(c.cfg(kvq)),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((c.T, Hq, d), 7.0, dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gq, gk, gv = c.parts(x)
    kvq.kvq_rope_append(c.cfg(kvq), kvq.rope(rot, inter), pool, gq, gk, gv, out, dev(cs), *c.places(), status=status)
    assert status.item() == 0
    got = out.cpu().numpy()
    assert np.array_equal(got[:n].view(np.uint16), qt.view(np.uint16))
    assert (got[n:] == 7).all()
    want = c.want_pool(kt, v[:n])
    assert np.array_equal(pool.cpu().numpy(), want)
    # in place, within the projection's rows; without queries
    kvq.kvq_rope_append(c.cfg(kvq), kvq.rope(rot, inter), pool.fill_(0xA5), gq, gk, gv, gq, dev(cs), *c.places())
    assert np.array_equal(c.parts(x.cpu().numpy())[0][:n].view(np.uint16), qt.view(np.uint16))
    assert np.array_equal(pool.cpu().numpy(), want)
    pool.fill_(0xA5)
    kvq.kvq_rope_append(c.cfg(kvq), kvq.rope(rot, inter), pool, None, gk, gv, None, dev(cs), *c.places())
    assert np.array_equal(pool.cpu().numpy(), want)
    # read back: as kvq_dequantize, sequence by sequence
    for dtype in (torch.float16, torch.float32):
        ok, ov = (torch.full((c.T, Hkv, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        kvq.kvq_dequantize_varlen(c.cfg(kvq), pool, *c.places(), ok, ov, status=status)
        for b, m in enumerate(new):
            if m:
                wk, wv = (torch.empty((m, Hkv, d), dtype=dtype, device="cuda") for _ in range(2))
                kvq.kvq_dequantize(c.cfg(kvq), pool, dev(c.table), b, start[b], m, wk, wv)
                lo = c.cu[b]
                assert torch.equal(ok[lo:lo + m], wk) and torch.equal(ov[lo:lo + m], wv)
        assert (ok[n:] == 7).all() and (ov[n:] == 7).all() and status.item() == 0


@pytest.mark.parametrize("rot,inter,sections", [(128, False, [24, 20, 20]), (64, True, [16, 16]), (128, True, [63, 0, 1]),
                                                (32, False, [7, 9])])
def test_rope_axes(kvq, rot, inter, sections):
    c = Batch(4, 2, 128, 16, 64, 128, [9, 40], [0, 100], seed=4)
    rng = np.random.default_rng(1)
    at = rng.integers(0, 500, (len(sections), c.T)).astype(np.int32)
    full = angles(500, rot)
    axis = np.repeat(np.arange(len(sections)), sections)
    cs = np.concatenate([full[at[axis], np.arange(rot // 2)[:, None]].T,
                         full[at[axis], rot // 2 + np.arange(rot // 2)[:, None]].T], axis=-1)
    q, k, v = c.parts(c.x)
    pool = torch.full((kvq.kvq_pool_bytes(c.cfg(kvq)),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.empty((c.T, 4, 128), dtype=torch.float16, device="cuda")
    gq, gk, gv = c.parts(dev(c.x))
    kvq.kvq_rope_append(c.cfg(kvq), kvq.rope(rot, inter, sections), pool, gq, gk, gv, out, dev(full), *c.places(),
                        positions=dev(at))
    assert np.array_equal(out.cpu().numpy().view(np.uint16), turned(q, cs, rot, inter).view(np.uint16))
    assert np.array_equal(pool.cpu().numpy(), c.want_pool(turned(k, cs, rot, inter), v))
    # one axis, positions of the caller's own
    cs = full[at[0]]
    kvq.kvq_rope_append(c.cfg(kvq), kvq.rope(rot, inter), pool, gq, gk, gv, out, dev(full), *c.places(), positions=dev(at[0]))
    assert np.array_equal(out.cpu().numpy().view(np.uint16), turned(q, cs, rot, inter).view(np.uint16))


def test_rope_append_nan_and_infinities_store_the_bytes_of_quantize_append(kvq):
    c = Batch(2, 2, 128, 16, 64, 128, [6], [0])
    for i, bad in enumerate((np.nan, np.inf, -np.inf)):
        c.x[i, 128 * (2 + i % 2) + 5], c.x[i, 128 * 4 + 70] = bad, bad
    full = np.zeros((8, 128), np.float32)
    full[:, :64] = 1.0  # no turn: k as it is (x * 1 - y * 0 keeps x unless y is not finite, as y = inf gives NaN)
    gq, gk, gv = c.parts(dev(c.x))
    pools = [torch.zeros(kvq.kvq_pool_bytes(c.cfg(kvq)), dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = torch.empty((6, 2, 128), dtype=torch.float16, device="cuda")
    kvq.kvq_rope_append(c.cfg(kvq), kvq.rope(128), pools[0], gq, gk, gv, out, dev(full), *c.places())
    kt = turned(c.parts(c.x)[1], full[:6], 128, False)
    kvq.kvq_quantize_append_varlen(c.cfg(kvq), pools[1], dev(kt), gv.contiguous(), *c.places())
    assert torch.equal(pools[0], pools[1])


def test_rope_append_bad_places_are_skipped_and_flagged(kvq):
    c = Batch(2, 2, 128, 16, 64, 128, [4, 4, 4], [0, 0, 30], seed=2)
    c.table[1, 0] = c.num_pages  # no such page
    c.table[2, :] = c.table[2, 0]
    bt = dev(c.table[:, :2].copy())  # positions 32, 33 of sequence 2 lie outside
    cs = angles(40, 128)
    q, k, v = c.parts(c.x)
    pool = torch.full((kvq.kvq_pool_bytes(c.cfg(kvq)),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((12, 2, 128), 7.0, dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gq, gk, gv = c.parts(dev(c.x))
    start, cu = dev(c.start, torch.int32), dev(c.cu)
    kvq.kvq_rope_append(c.cfg(kvq), kvq.rope(128), pool, gq, gk, gv, out, dev(cs), bt, start, cu, status=status)
    assert status.item() == kvq.KVQ_FLAG_BAD_PAGE | kvq.KVQ_FLAG_BAD_POSITION
    kt = turned(k, cs[c.pos], 128, False)
    assert np.array_equal(out.cpu().numpy(), turned(q, cs[c.pos], 128, False))  # q turns all the same
    c.new = [4, 0, 2]
    assert np.array_equal(pool.cpu().numpy(), c.want_pool(kt, v))
    # read back: zero rows outside the table, page 0 for the bad page
    status.zero_()
    ok, ov = (torch.full((12, 2, 128), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    kvq.kvq_dequantize_varlen(c.cfg(kvq), pool, bt, start, cu, ok, ov, status=status)
    assert status.item() == kvq.KVQ_FLAG_BAD_PAGE | kvq.KVQ_FLAG_BAD_POSITION
    assert not ok[10:].any() and not ov[10:].any() and ok[8:10].any()
    # a row whose angle is missing is skipped whole
    status.zero_()
    before, out2 = pool.clone(), torch.full((12, 2, 128), 7.0, dtype=torch.float16, device="cuda")
    at = torch.full((12,), 40, dtype=torch.int32, device="cuda")
    at[1] = -1
    kvq.kvq_rope_append(c.cfg(kvq), kvq.rope(128), pool, gq, gk, gv, out2, dev(cs), bt, start, cu, positions=at,
                        status=status)
    assert status.item() == kvq.KVQ_FLAG_BAD_POSITION and torch.equal(pool, before) and (out2 == 7).all()


def test_many_sequences(kvq):
    new = [int(x) for x in np.random.default_rng(0).integers(0, 3, 2100)]
    c = Batch(1, 1, 64, 16, 32, 32, new, [b % 40 for b in range(2100)], pad=5, seed=3)
    cs = angles(64, 64)
    q, k, v = c.parts(c.x)
    n = c.cu[-1]
    pool = torch.full((kvq.kvq_pool_bytes(c.cfg(kvq)),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.zeros((c.T, 1, 64), dtype=torch.float16, device="cuda")
    gq, gk, gv = c.parts(dev(c.x))
    kvq.kvq_rope_append(c.cfg(kvq), kvq.rope(64), pool, gq, gk, gv, out, dev(cs), *c.places())
    assert np.array_equal(out.cpu().numpy()[:n], turned(q[:n], cs[c.pos], 64, False))
    assert np.array_equal(pool.cpu().numpy(), c.want_pool(turned(k[:n], cs[c.pos], 64, False), v[:n]))


def latent_rows(x, gain, eps, L, G):
    """What fp16 rows x [n, L] hold once normalised and quantized: (codes, fp16 scales), as the header defines."""
    y = x.astype(np.float32)
    if gain is not None:
        r = (1.0 / np.sqrt((x.astype(np.float64) ** 2).mean(-1, keepdims=True) + np.float64(np.float32(eps)))).astype(np.float32)
        y = (y * r) * gain
    g = y.reshape(len(x), L // G, G)
    s = (np.abs(g).max(-1) / np.float32(7)).astype(np.float16)
    s[s == 0] = 1
    codes = np.clip(np.rint(g / s.astype(np.float32)[..., None]), -7, 7).astype(np.int32)
    return codes.reshape(len(x), L), s


@pytest.mark.parametrize("L,G,P,H,inter,norm", [(512, 64, 64, 16, True, True), (512, 128, 16, 5, False, True),
                                                (256, 32, 32, 1, True, False), (256, 128, 64, 33, False, True),
                                                (512, 32, 16, 0, False, False)])
@pytest.mark.parametrize("new,start,pad", [([1, 1, 1], [0, 63, 100], 0), ([70, 0, 3, 200], [5, 0, 64, 31], 9)])
def test_latent_append(kvq, L, G, P, H, inter, norm, new, start, pad):
    rng = np.random.default_rng(L + G)
    cu, T = ragged(new, pad)
    n, R = cu[-1], 64
    x = rng.standard_normal((T, L + R + 8)).astype(np.float16)
    x[:, :3] *= np.float16(20)
    x[0, :L] = 0 if not norm else x[0, :L] * np.float16(2.0 ** -9)
    x[1, :L] = (np.sign(x[1, :L]) * 50000).astype(np.float16)
    gain = (1 + 0.2 * rng.standard_normal(L)).astype(np.float32) if norm else None
    pages = [(s + m + P - 1) // P for s, m in zip(start, new)]
    num_pages = sum(pages) + 1
    order = rng.permutation(num_pages).astype(np.int32)
    table = np.full((len(new), max(pages)), -1, np.int32)
    at = 0
    for b, m in enumerate(pages):
        table[b, :m] = order[at:at + m]
        at += m
    cfg, cs = kvq.latent_config(L, R, P, G, num_pages), angles(400, R)
    pool = torch.full((kvq.kvq_latent_pool_bytes(cfg),), 0xA5, dtype=torch.uint8, device="cuda")
    qpe, qin = (rng.standard_normal((T, max(H, 1), w)).astype(np.float16) for w in (R, L + R))
    gx, q = dev(x), dev(qin)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    places = dev(table), dev(start, torch.int32), dev(cu)
    kvq.kvq_latent_append(cfg, kvq.rope(R, inter), pool, gx[:, :L + R], None if gain is None else dev(gain), 1e-5,
                          dev(qpe) if H else None, q if H else None, dev(cs), *places, status=status)
    assert status.item() == 0
    seq = np.repeat(np.arange(len(new)), new)
    pos = np.asarray(start)[seq] + np.arange(n) - cu[seq]
    codes, s = latent_rows(x[:n, :L], gain, 1e-5, L, G)
    key = turned(x[:n, None, L:L + R], cs[pos], R, inter)[:, 0]
    want = np.full((num_pages, P * (L // 2 + 2 * (L // G) + 2 * R)), 0xA5, np.uint8)
    page, slot = table[seq, pos // P], pos % P
    nib = (codes + 8).astype(np.uint8)
    for off, row, part in ((0, L // 2, nib[:, 0::2] | nib[:, 1::2] << 4), (P * L // 2, 2 * (L // G), s.view(np.uint8)),
                           (P * (L // 2 + 2 * (L // G)), 2 * R, key.view(np.uint8))):
        want[page[:, None], off + slot[:, None] * row + np.arange(row)] = part
    assert np.array_equal(pool.cpu().numpy(), want.reshape(-1))
    if H:
        qin[:n, :, L:] = turned(qpe[:n], cs[pos], R, inter)
        assert np.array_equal(q.cpu().numpy().view(np.uint16), qin.view(np.uint16))
    # read back
    out = torch.full((T, L + R), 7.0, dtype=torch.float16, device="cuda")
    kvq.kvq_latent_dequantize(cfg, pool, *places, out, status=status)
    got = out.cpu().numpy()
    vals = (codes.astype(np.float32) * np.repeat(s.astype(np.float32), G, axis=-1)).astype(np.float16)
    assert np.array_equal(got[:n], np.concatenate([vals, key], axis=-1)) and (got[n:] == 7).all() and status.item() == 0


def test_latent_rows_bad_places(kvq):
    cfg, cs = kvq.latent_config(256, 64, 16, 64, 3), dev(angles(64, 64))
    x = torch.randn(6, 320, device="cuda").half()
    pool = torch.full((kvq.kvq_latent_pool_bytes(cfg),), 0xA5, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    table, cu = dev([[0], [9]], torch.int32), dev([0, 3, 6], torch.int32)
    start = dev([14, 0], torch.int32)  # position 16 lies outside the table; sequence 1 has no page
    kvq.kvq_latent_append(cfg, kvq.rope(64), pool, x, None, 0.0, None, None, cs, table, start, cu, status=status)
    assert status.item() == kvq.KVQ_FLAG_BAD_PAGE | kvq.KVQ_FLAG_BAD_POSITION
    touched = (pool.view(3, -1) != 0xA5).any(-1)
    assert touched.tolist() == [True, False, False]
    status.zero_()
    out = torch.full((6, 320), 7.0, dtype=torch.float16, device="cuda")
    kvq.kvq_latent_dequantize(cfg, pool, table, start, cu, out, status=status)
    assert status.item() == kvq.KVQ_FLAG_BAD_PAGE | kvq.KVQ_FLAG_BAD_POSITION
    assert not out[2].any() and (out[:2] != 7).any()
    # no angle for position 64
    status.zero_()
    before = pool.clone()
    kvq.kvq_latent_append(cfg, kvq.rope(64), pool, x, None, 0.0, None, None, cs, table, start, cu,
                          positions=torch.full((6,), 64, dtype=torch.int32, device="cuda"), status=status)
    assert status.item() == kvq.KVQ_FLAG_BAD_POSITION and torch.equal(pool, before)
