"""Attention of ragged batches of rows over the INT4 cache and over the latent cache, against fp64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from conftest import cuda_available
from eviction_testlib import Pool
from rows_testlib import LatentPool, attend64, ragged

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_q(T, H, n, seed=0, size=1.0):
    return (size * np.random.default_rng(seed).standard_normal((T, H, n))).astype(np.float16)


class Chunk:
    """A case of kvq_chunk_attention: sequences of `total` positions whose last `new` rows attend."""

    def __init__(self, kvq, Hkv, r, d, P, Gk, Gv, new, total, pad=0, seed=0, blocks=None, size=1.0):
        self.kvq, self.new, self.total, self.r = kvq, new, total, r
        self.pool = Pool("int4", Hkv, d, total, P, Gk, Gv, seed=seed, poison=True, blocks=blocks)
        self.cu, self.T = ragged(new, pad)
        self.q = make_q(self.T, Hkv * r, d, seed, size)
        self.cfg, self.max_len, self.scale = self.pool.cfg(kvq), max(max(total), 1), d ** -0.5
        self.ws = kvq.new_chunk_workspace(self.cfg, len(new), Hkv * r, self.max_len)
        self.out = torch.full((self.T, Hkv * r, d), 7.0, dtype=torch.float16, device="cuda")
        self.args = [self.pool.gpu(), dev(self.q), self.pool.table_gpu(), ints(total), ints(self.cu)]

    def run(self, **k):
        pool, q, table, lens, cu = self.args
        self.kvq.kvq_chunk_attention(self.cfg, pool, q, table, lens, cu, self.max_len, self.scale, self.out, self.ws, **k)
        return self.out

    def check(self, rows=None, flags=0):
        assert self.kvq.kvq_read_status(self.ws) == flags
        check_rows(self, lambda b, n: [(K, V) for K, V in zip(*self.pool.values(b, n))], self.r, rows)


class Latent:
    """A case of kvq_latent_attention."""

    def __init__(self, kvq, L, H, P, G, new, total, pad=0, seed=0, size=1.0):
        self.kvq, self.new, self.total, self.H = kvq, new, total, H
        self.pool = LatentPool(L, total, P, G, seed=seed)
        self.cu, self.T = ragged(new, pad)
        self.q = make_q(self.T, H, L + 64, seed, size)
        self.cfg, self.max_len, self.scale = self.pool.cfg(kvq), max(max(total), 1), 0.5 * (L + 64) ** -0.5
        self.ws = kvq.new_latent_workspace(self.cfg, len(new), H, self.max_len)
        self.out = torch.full((self.T, H, L), 7.0, dtype=torch.float16, device="cuda")
        self.args = [self.pool.gpu(), dev(self.q), self.pool.table_gpu(), ints(total), ints(self.cu)]

    def run(self, **k):
        pool, q, table, lens, cu = self.args
        self.kvq.kvq_latent_attention(self.cfg, pool, q, table, lens, cu, self.max_len, self.scale, self.out, self.ws, **k)
        return self.out

    def check(self, rows=None, flags=0):
        assert self.kvq.kvq_read_status(self.ws) == flags
        check_rows(self, lambda b, n: [(x, x[:, :self.pool.L]) for x in [self.pool.rows(b, n)]], self.H, rows)


def check_rows(c, cache, r, rows):
    """Every row (or those at the offsets `rows` picks of a sequence's n) of every sequence against fp64."""
    got, q = c.out.cpu().numpy().astype(np.float64), c.q.astype(np.float64)
    assert (got[c.cu[-1]:] == 7).all(), "rows behind the last sequence"
    for b, (m, n) in enumerate(zip(c.new, c.total)):
        if m == 0:
            continue
        pick = range(m) if rows is None else sorted({i % m for i in rows})
        kv = cache(b, n)
        for h in range(q.shape[1]):
            K, V = kv[h // r]
            for i in pick:
                at = c.cu[b] + i
                want, tol = attend64(q[at:at + 1, h], K, V, n - m + i, c.scale)
                err = np.abs(got[at, h] - want[0])
                assert (err <= tol[0]).all(), (b, h, i, float(err.max()), float(tol[0].min()))


CHUNKS = [  # Hkv, r, d, P, Gk, Gv, new, total
    (2, 4, 128, 16, 64, 128, [1], [1]),
    (1, 1, 128, 16, 64, 64, [1, 2, 0, 3], [1, 2, 5, 300]),
    (2, 1, 128, 64, 128, 128, [130], [130]),
    (1, 8, 128, 32, 32, 32, [17, 16, 33], [17, 400, 129]),
    (2, 3, 128, 16, 32, 64, [43, 1], [171, 128]),
    (1, 5, 64, 16, 64, 32, [60, 9], [60, 1000]),
    (3, 2, 64, 32, 32, 64, [129, 0, 7], [257, 0, 127]),
    (1, 7, 64, 64, 32, 32, [37], [4000]),
    (1, 6, 128, 16, 128, 32, [22, 21], [255, 256]),
    (2, 4, 128, 16, 64, 128, [8, 8], [3001, 4097]),
    (1, 2, 128, 16, 64, 128, [513], [900]),
]


@pytest.mark.parametrize("Hkv,r,d,P,Gk,Gv,new,total", CHUNKS)
def test_chunk(kvq, Hkv, r, d, P, Gk, Gv, new, total):
    c = Chunk(kvq, Hkv, r, d, P, Gk, Gv, new, total, pad=2, seed=d + r)
    c.run()
    c.check()
    first = c.out.clone()
    c.ws[256:].fill_(0xFF)  # nothing in a workspace has to be kept
    assert torch.equal(c.run(), first)


LATENTS = [  # L, H, P, G, new, total
    (512, 16, 64, 64, [1], [1]),
    (512, 1, 16, 32, [1, 1, 0, 2], [1, 700, 9, 130]),
    (512, 128, 64, 64, [1, 1], [129, 513]),
    (256, 20, 16, 32, [3, 13, 1], [3, 300, 128]),
    (512, 33, 32, 128, [2, 5], [64, 333]),
    (256, 7, 64, 128, [40], [1111]),
    (512, 64, 16, 64, [3], [127]),
    (256, 100, 32, 64, [2], [257]),
]


@pytest.mark.parametrize("L,H,P,G,new,total", LATENTS)
def test_latent(kvq, L, H, P, G, new, total):
    c = Latent(kvq, L, H, P, G, new, total, pad=3, seed=L + H)
    c.run()
    c.check()
    first = c.out.clone()
    c.ws[256:].fill_(0xFF)
    assert torch.equal(c.run(), first)


def both(kvq, new, total, **k):
    return [Chunk(kvq, 2, 4, 128, 16, 64, 128, new, total, **k), Latent(kvq, 512, 16, 64, 64, new, total, **k)]


def test_long_sequences_split_over_the_device(kvq):
    for c in both(kvq, [1, 3], [40001, 17000]):
        c.run()
        c.check()


def test_a_prompt_larger_than_the_grid(kvq):
    c = Chunk(kvq, 4, 4, 128, 16, 64, 128, [3000, 1500], [3000, 2500])
    c.run()
    c.check(rows=[0, 1, 31, 32, 63, 64, 65, 127, 128, 700, 1499, 2047, 2998, 2999])
    c = Latent(kvq, 512, 16, 64, 64, [500, 100], [500, 2500])
    c.run()
    c.check(rows=[0, 1, 3, 4, 5, 99, 127, 128, 250, 498, 499])


def test_large_scores_and_sharp_softmax(kvq):
    for c in both(kvq, [20, 1], [500, 1500], size=30.0):
        c.run()
        c.check(rows=[0, 7, 19])


@pytest.mark.parametrize("d,r", [(128, 4), (64, 1), (64, 7)])
def test_a_prompt_among_single_tokens(kvq, d, r):
    """Few lines a sequence on average, one of them with many: items of one sequence share its tiles, and the last is short."""
    new = [0, 1, 97 if r < 7 else 41, 1, 1] + [1] * 11
    total = [3, 1, 650, 128, 129] + [40 * i + 1 for i in range(11)]
    assert sum(new) * r <= 32 * len(new)
    c = Chunk(kvq, 2, r, d, 32, 32, 64, new, total, pad=3, seed=r)
    c.run()
    c.check()


@pytest.mark.parametrize("case", ["few", "many", "latent"])
def test_enormous_scores_pick_one_position(kvq, case):
    """Scores of 2^30 and more: the softmax is 1 at the largest.  Rows whose two largest are closer than four times what
    the scores may be off by are left out.  The weight is rounded to fp16, so are the value and the output: half a step each."""
    new, total = [3, 1, 2], [3, 129, 700]
    if case == "latent":
        c = Latent(kvq, 256, 5, 32, 64, new, total, seed=3, size=1000.0)
    else:
        c = Chunk(kvq, 2, 2, 128, 16, 64, 128, new if case == "few" else [150, 40], total if case == "few" else [700, 40],
                  seed=3, size=1000.0)
    c.scale = 65536.0
    got = c.run().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all() and kvq.kvq_read_status(c.ws) == 0
    q, seen, clear, largest = c.q.astype(np.float64), 0, 0, 0.0
    for b, (m, n) in enumerate(zip(c.new, c.total)):
        kv = [(x, x[:, :c.pool.L]) for x in [c.pool.rows(b, n)]] if case == "latent" else list(zip(*c.pool.values(b, n)))
        for h in range(q.shape[1]):
            K, V = kv[0] if case == "latent" else kv[h // c.r]
            for i in range(m):
                end = n - m + i + 1
                z = K[:end] @ q[c.cu[b] + i, h] * c.scale
                dz = (np.abs(K[:end]) @ np.abs(q[c.cu[b] + i, h])).max() * c.scale * (2.0 ** -11 + K.shape[1] * 2.0 ** -23)
                top, seen, largest = int(z.argmax()), seen + 1, max(largest, float(z.max()))
                if end > 1 and np.sort(z)[-1] - np.sort(z)[-2] < 4 * dz:
                    continue
                clear += 1
                err = np.abs(got[c.cu[b] + i, h] - V[top])
                assert (err <= 3.2 * 2.0 ** -11 * np.abs(V[top]) + 2.0 ** -24).all(), (b, h, i, float(err.max()))
    assert 2 * clear > seen and largest > 2.0 ** 30


def test_negative_scale(kvq):
    for c in both(kvq, [5], [300]):
        c.scale = -c.scale
        c.run()
        c.check()


def test_rows_before_the_first_position_are_zeros(kvq):
    for c in both(kvq, [9, 4, 200], [5, 0, 3]):
        out = c.run()
        assert not out[:4].any() and not out[9:13].any() and not out[13:210].any()
        c.check()


def test_many_sequences(kvq):
    rng = np.random.default_rng(5)
    new = [int(x) for x in rng.integers(0, 3, 1500)]
    total = [n + int(x) for n, x in zip(new, rng.integers(0, 40, 1500))]
    for c in (Chunk(kvq, 1, 2, 64, 16, 32, 64, new, total), Latent(kvq, 256, 4, 16, 64, new, total)):
        c.run()
        c.check()


def test_one_row_agrees_with_decode_attention(kvq):
    c = Chunk(kvq, 4, 4, 128, 16, 64, 128, [1, 1, 1], [1, 777, 5000])
    c.run()
    pool, q, table, lens, _ = c.args
    out = torch.empty((3, 16, 128), dtype=torch.float32, device="cuda")
    kvq.kvq_decode_attention(c.cfg, pool, q, table, lens, c.max_len, c.scale, out,
                             kvq.new_workspace(c.cfg, 3, 16, c.max_len))
    for b, n in enumerate(c.total):
        for h in range(16):
            K, V = (x[h // 4] for x in c.pool.values(b, n))
            _, tol = attend64(c.q[b:b + 1, h].astype(np.float64), K, V, n - 1, c.scale)
            err = (c.out[b, h].double() - out[b, h].double()).abs().cpu().numpy()
            assert (err <= tol[0] + 2e-6 * np.abs(V).max()).all()


def test_lengths_beyond_the_bound_are_cut_and_flagged(kvq):
    for c in both(kvq, [3], [100]):
        c.max_len = 70  # rows at positions 67 .. 69
        c.run()
        c.total = [70]
        c.check(flags=kvq.KVQ_FLAG_BAD_POSITION)
    for c in both(kvq, [3], [100]):  # one page short of the sequence
        pages = (100 + c.pool.P - 1) // c.pool.P - 1
        c.args[2] = c.args[2][:, :pages].contiguous()
        c.run()
        c.total = [pages * c.pool.P]
        c.check(flags=kvq.KVQ_FLAG_BAD_POSITION)


def test_negative_lengths_are_empty(kvq):
    for c in both(kvq, [3], [100]):
        c.args[3] = ints([-5])
        assert not c.run().any() and kvq.kvq_read_status(c.ws) == 0


def test_bad_pages_read_as_page_0_and_are_flagged(kvq):
    for c in both(kvq, [4], [300]):
        good = c.args[2].clone()
        for bad in (-1, c.pool.num_pages, 1 << 30, -(1 << 31)):
            c.ws[:256].zero_()
            c.args[2] = good.clone()
            c.args[2][0, 2] = bad
            got = c.run().clone()
            assert kvq.kvq_read_status(c.ws) == kvq.KVQ_FLAG_BAD_PAGE
            c.args[2][0, 2] = 0
            assert torch.equal(c.run().view(torch.int16), got.view(torch.int16))  # (page 0 may hold NaN)


def test_offsets_that_do_not_ascend_stay_inside(kvq):
    for c in both(kvq, [4, 4, 4], [300, 20, 50]):
        for cu in ([0, 9, 3, 12], [5, 5, 5, 5], [-3, 4, 8, 12], [12, 8, 4, 0], [0, 4, 8, 1 << 30], [0, -5, 1 << 30, 12]):
            c.args[4] = ints(cu)
            c.run()
            torch.cuda.synchronize()
        c.args[4] = ints(c.cu)
        c.run()
        c.check()


def test_pool_beyond_4_gb(kvq):
    """Pages whose bytes lie beyond 32-bit offsets."""
    for c in both(kvq, [3], [200]):
        block = len(c.pool.bytes.reshape(-1)) // c.pool.num_pages
        pages = (1 << 32) // block + 2 + c.pool.num_pages
        far = torch.empty(pages * block, dtype=torch.uint8, device="cuda")
        shift = pages - c.pool.num_pages
        far[shift * block:] = c.args[0]
        want = c.run().clone()
        c.cfg.num_pages = pages
        c.args[0] = far
        c.args[2] = torch.where(c.args[2] >= 0, c.args[2] + shift, c.args[2])
        c.out.fill_(7)
        assert torch.equal(c.run(), want)
        del far


def test_graph_and_streams(kvq):
    """A captured call replayed with new lengths and rows, on a stream of its own; two graphs share a workspace."""
    for c in both(kvq, [8, 2], [600, 301], pad=6):
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graphs = []
        with torch.cuda.stream(stream):
            c.run()
            for _ in range(2):
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=stream):
                    c.run()
                graphs.append(g)
            c.out.fill_(7)
            graphs[0].replay()
            graphs[1].replay()
        stream.synchronize()
        c.check()
        c.new, c.total = [1, 12], [599, 300]
        c.cu, _ = ragged(c.new)
        with torch.cuda.stream(stream):
            c.args[3].copy_(ints(c.total))
            c.args[4].copy_(ints(c.cu))
            c.out.fill_(7)
            graphs[0].replay()
        stream.synchronize()
        c.check()
        c.out.fill_(7)
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        c.run(stream=other)
        other.synchronize()
        c.check()


def test_binding_refuses(kvq):
    for c in both(kvq, [3], [100]):
        pool, q, table, lens, cu = c.args
        fn = kvq.kvq_chunk_attention if isinstance(c, Chunk) else kvq.kvq_latent_attention
        for bad in (dict(q=q.float()), dict(q=q[:, :, :-8]), dict(q=q.cpu()), dict(q=q.transpose(0, 1)), dict(lens=lens.long()),
                    dict(lens=ints([1, 2])), dict(cu=ints([0])), dict(cu=cu.cpu()), dict(out=c.out.float()),
                    dict(out=c.out[:2]), dict(table=table[0]), dict(pool=pool[:-1]), dict(pool=pool.cpu())):
            a = dict(pool=pool, q=q, table=table, lens=lens, cu=cu, out=c.out)
            a.update(bad)
            with pytest.raises((ValueError, kvq.KvqError)):
                fn(c.cfg, a["pool"], a["q"], a["table"], a["lens"], a["cu"], c.max_len, c.scale, a["out"], c.ws)
        with pytest.raises(kvq.KvqError) as e:
            fn(c.cfg, pool, q, table, lens, cu, c.max_len, c.scale, c.out, c.ws[:128])
        assert e.value.code == kvq.KVQ_EWORKSPACE
