"""Decode attention with accumulated position weights, the selection by them and the compaction, against fp64 and
plain numpy; the three together as a serving loop runs them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from conftest import cuda_available
from eviction_testlib import EPS32, Pool, errors, score_error, softmax64

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]


def make_q(B, Hq, d, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((B, Hq, d)).astype(np.float16)).cuda()


def call_weights(kvq, pool, x, q, decay, weights, max_len=None, ws=None, lens=None, stream=None):
    cfg = pool.cfg(kvq)
    B, Hq, d = q.shape
    max_len = max(pool.lens) if max_len is None else max_len
    new, fn = (kvq.new_int8_weights_workspace, kvq.kvq_int8_decode_attention_weights) if pool.codec == "int8" else \
        (kvq.new_weights_workspace, kvq.kvq_decode_attention_weights)
    ws = new(cfg, B, Hq, max_len) if ws is None else ws
    out = torch.full((B, Hq, d), float("nan"), device="cuda")
    fn(cfg, x, q, pool.table_gpu(), pool.lens_gpu() if lens is None else lens, max_len, d ** -0.5, decay, weights, out,
       ws, stream=stream)
    return out, ws


def check_weights(pool, q, decay, before, out, after, lens=None):
    """out and the updated weights against fp64, each within its derived bound."""
    q = q.cpu().numpy().astype(np.float64)
    out, before, after = out.cpu().numpy(), before.cpu().numpy(), after.cpu().numpy()
    B, Hq, d = q.shape
    r = Hq // pool.Hkv
    for b, n in enumerate(pool.lens if lens is None else lens):
        assert np.array_equal(after[b, :, n:], before[b, :, n:], equal_nan=True), "positions behind the sequence"
        if n == 0:
            assert not out[b].any()
            continue
        K, V = pool.values(b, n)
        for h in range(pool.Hkv):
            qh = q[b, h * r:(h + 1) * r]
            z = qh @ K[h].T * d ** -0.5
            dz = score_error(qh, K[h], d ** -0.5)
            p = softmax64(z)
            mass, slack = np.zeros(n), np.zeros(n)
            for g in range(r):
                tol, rel = errors(z[g], V[h], dz, pool.codec)
                err = np.abs(out[b, h * r + g] - p[g] @ V[h])
                assert err.max() <= tol, (b, h, g, err.max(), tol)
                mass += p[g]
                slack += rel * p[g]
            want = mass if decay == 0.0 else decay * before[b, h, :n].astype(np.float64) + mass
            slack += 2 * (r + 2) * EPS32 * np.abs(want) + 1e-37
            assert (np.abs(after[b, h, :n] - want) <= slack).all(), (b, h, np.max(np.abs(after[b, h, :n] - want) / slack))


@pytest.mark.parametrize("Hkv,r,d,P,Gk,Gv,lens", [
    (8, 1, 128, 16, 64, 128, [513]),                     # four kv heads a unit
    (3, 1, 128, 16, 64, 64, [1, 0, 16, 17, 700]),        # one head a unit, one query head
    (4, 2, 128, 16, 32, 32, [15, 33, 1024]),             # two heads a unit
    (6, 2, 64, 16, 64, 32, [5, 700, 0]),
    (3, 2, 128, 16, 128, 64, [200, 1]),
    (2, 4, 128, 16, 128, 128, [2049, 5]),
    (2, 5, 128, 16, 64, 128, [300, 31]),                 # two slots a thread, three of them empty
    (1, 8, 128, 16, 64, 32, [777]),
    (2, 3, 128, 32, 64, 128, [64, 65, 999]),
    (4, 1, 128, 64, 64, 128, [63, 128, 1]),
    (2, 8, 128, 64, 128, 64, [500, 0]),
    (4, 1, 64, 16, 32, 64, [255, 1]),
    (2, 7, 64, 32, 64, 32, [400]),
    (2, 4, 256, 16, 64, 128, [300, 17]),
    (3, 1, 256, 64, 128, 32, [129, 0, 640]),
])
@pytest.mark.parametrize("decay", [1.0, 0.0, 0.75])
def test_attention_and_weights_match_fp64(kvq, Hkv, r, d, P, Gk, Gv, lens, decay):
    pool = Pool("int4", Hkv, d, lens, P, Gk, Gv, seed=d + r, poison=True)
    q = make_q(len(lens), Hkv * r, d, 3)
    before = torch.rand(len(lens), Hkv, max(lens) + 5, device="cuda")
    if decay == 0.0:
        before.fill_(float("nan"))  # not read
    weights = before.clone()
    out, ws = call_weights(kvq, pool, pool.gpu(), q, decay, weights)
    assert kvq.kvq_read_status(ws) == 0
    check_weights(pool, q, decay, before, out, weights)


@pytest.mark.parametrize("Hkv,r,P,lens", [(4, 1, 16, [1, 0, 513]), (2, 4, 64, [64, 700]), (2, 6, 32, [33, 250]),
                                          (1, 8, 16, [1025])])
def test_int8_attention_and_weights_match_fp64(kvq, Hkv, r, P, lens):
    pool = Pool("int8", Hkv, 128, lens, P, 128, 128, seed=r, poison=True)
    q = make_q(len(lens), Hkv * r, 128, 4)
    before = torch.rand(len(lens), Hkv, max(lens), device="cuda")
    weights = before.clone()
    out, ws = call_weights(kvq, pool, pool.gpu(), q, 0.5, weights)
    assert kvq.kvq_read_status(ws) == 0
    check_weights(pool, q, 0.5, before, out, weights)


def test_many_sequences_and_a_long_one(kvq):
    # over 256 sequences the combine reads the published page prefix
    lens = [(7 * b) % 40 for b in range(300)] + [9000]
    pool = Pool("int4", 2, 64, lens, 16, 32, 64, seed=9)
    q = make_q(len(lens), 4, 64, 5)
    before = torch.rand(len(lens), 2, max(lens), device="cuda")
    weights = before.clone()
    out, ws = call_weights(kvq, pool, pool.gpu(), q, 1.0, weights)
    assert kvq.kvq_read_status(ws) == 0
    check_weights(pool, q, 1.0, before, out, weights)


def test_equal_bits_on_repeat_side_stream_and_replayed_graph(kvq):
    pool = Pool("int4", 4, 128, [600, 77], 16, 64, 128, seed=2)
    x, q = pool.gpu(), make_q(2, 16, 128, 6)
    start = torch.rand(2, 4, 600, device="cuda")
    w0 = start.clone()
    out0, ws = call_weights(kvq, pool, x, q, 0.5, w0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w1 = start.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out1, _ = call_weights(kvq, pool, x, q, 0.5, w1)
    side.synchronize()
    assert torch.equal(out0, out1) and torch.equal(w0, w1)
    w2, out2 = start.clone(), torch.empty_like(out0)
    table, lens, cfg = pool.table_gpu(), pool.lens_gpu(), pool.cfg(kvq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_decode_attention_weights(cfg, x, q, table, lens, 600, 128 ** -0.5, 0.5, w2, out2, ws)
    for _ in range(2):
        w2.copy_(start)
        graph.replay()
        assert torch.equal(out0, out2) and torch.equal(w0, w2)


def test_two_graphs_share_a_workspace(kvq):
    pools = [Pool("int4", 4, 128, [600, 77], 16, 64, 128, seed=2), Pool("int4", 4, 128, [31, 400], 16, 64, 128, seed=3)]
    cfg = [p.cfg(kvq) for p in pools]
    ws = kvq.new_weights_workspace(cfg[0], 2, 16, 600)
    sets, graphs, want = [], [], []
    for p, c in zip(pools, cfg):
        s = (p.gpu(), make_q(2, 16, 128, 6), p.table_gpu(), p.lens_gpu(), torch.zeros(2, 4, 600, device="cuda"),
             torch.empty(2, 16, 128, device="cuda"))

        def go(c=c, s=s):
            kvq.kvq_decode_attention_weights(c, *s[:4], 600, 128 ** -0.5, 0.0, s[4], s[5], ws)

        go()
        want.append((s[4].clone(), s[5].clone()))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go()
        sets.append(s)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0):
        sets[i][4].zero_()
        sets[i][5].zero_()
        graphs[i].replay()
        assert torch.equal(sets[i][4], want[i][0]) and torch.equal(sets[i][5], want[i][1])


@pytest.mark.parametrize("codec", ["int4", "int8"])
def test_thousands_of_short_sequences(kvq, codec):
    # segments of one page, many to a CTA: warps without units of a segment keep up with the others
    lens = [1 + (7 * b) % 40 for b in range(2100)]
    pool = Pool(codec, 1, 128, lens, 64 if codec == "int8" else 16, 64, 128, seed=9)
    q = make_q(len(lens), 3, 128, 5)
    before = torch.zeros(len(lens), 1, 40, device="cuda")
    weights = before.clone()
    out, ws = call_weights(kvq, pool, pool.gpu(), q, 1.0, weights)
    assert kvq.kvq_read_status(ws) == 0
    check_weights(pool, q, 1.0, before, out, weights)


def test_pool_beyond_four_gigabytes(kvq):
    """Pages whose byte offsets pass 32 bits: attention with weights, differential attention and compaction give what
    the same pages give at the start of a small pool."""
    pool = Pool("int4", 2, 128, [100, 60], 16, 64, 128, seed=8)
    small, q = pool.gpu(), make_q(2, 4, 128, 3)
    pages = 5 * 2 ** 30 // (2 * pool.block)
    shift = pages - pool.num_pages
    big_cfg = kvq.config(2, 128, 16, 64, 128, pages)
    big = torch.zeros(kvq.kvq_pool_bytes(big_cfg), dtype=torch.uint8, device="cuda")
    big[-small.numel():] = small
    table = pool.table_gpu()
    far = torch.where(table >= 0, table + shift, table)
    kept = torch.from_numpy(random_kept(pool, 30, 2)).cuda()
    lam = torch.tensor([0.1, 0.5, 0.7, 0.9], device="cuda")

    def go(cfg, x, t):
        w, out, o2 = torch.zeros(2, 2, 100, device="cuda"), torch.empty(2, 4, 128, device="cuda"), \
            torch.empty(2, 4, 128, device="cuda")
        kvq.kvq_decode_attention_weights(cfg, x, q, t, pool.lens_gpu(), 100, 0.1, 1.0, w, out,
                                         kvq.new_weights_workspace(cfg, 2, 4, 100))
        kvq.kvq_diff_decode_attention(cfg, x, q, t, pool.lens_gpu(), 100, 0.1, lam, None, 0.0, 1.0, o2,
                                      kvq.new_diff_workspace(cfg, 2, 4, 100))
        kvq.kvq_evict_compact(cfg, x, t, t, pool.lens_gpu(), kept, w)
        return w, out, o2

    want, got = go(pool.cfg(kvq), small, table), go(big_cfg, big, far)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.equal(big[-small.numel():], small) and not big[:-small.numel()].any()


def test_agrees_with_plain_decode_attention(kvq):
    pool = Pool("int4", 8, 128, [1000, 3], 16, 64, 128, seed=12)
    x, q, cfg = pool.gpu(), make_q(2, 8, 128, 7), pool.cfg(kvq)
    out, _ = call_weights(kvq, pool, x, q, 1.0, torch.zeros(2, 8, 1000, device="cuda"))
    plain = torch.empty_like(out)
    kvq.kvq_decode_attention(cfg, x, q, pool.table_gpu(), pool.lens_gpu(), 1000, 128 ** -0.5, plain,
                             kvq.new_workspace(cfg, 2, 8, 1000))
    # both are within 2e-4 of the exact result, the framework's tolerance of decode attention
    assert (out - plain).abs().max().item() <= 4e-4


def test_step_is_append_then_attention(kvq):
    for Hkv, r, d, P in ((8, 1, 128, 16), (2, 4, 128, 32), (2, 3, 256, 16), (4, 2, 128, 16), (2, 2, 64, 16)):
        pool = Pool("int4", Hkv, d, [64, 17, 200], P, 64, 64, seed=21, spare=4, blocks=16)
        x1, q, cfg = pool.gpu(), make_q(3, Hkv * r, d, 8), pool.cfg(kvq)
        x2 = x1.clone()
        k, v = make_q(3, Hkv, d, 30), make_q(3, Hkv, d, 31)
        pos = torch.tensor([63, 16, -1], dtype=torch.int32, device="cuda")  # the last sequence appends nothing
        start = torch.rand(3, Hkv, 200, device="cuda")
        w1, w2 = start.clone(), start.clone()
        ws = kvq.new_weights_workspace(cfg, 3, Hkv * r, 200)
        o1, o2 = torch.empty_like(q, dtype=torch.float32), torch.empty_like(q, dtype=torch.float32)
        kvq.kvq_decode_step_weights(cfg, x1, k, v, pos, q, pool.table_gpu(), pool.lens_gpu(), 200, d ** -0.5, 1.0, w1,
                                    o1, ws)
        for b in (0, 1):
            kvq.kvq_quantize_append(cfg, x2, k[b:b + 1, None].contiguous(), v[b:b + 1, None].contiguous(),
                                    pool.table_gpu()[b:b + 1].contiguous(), pos[b:b + 1].contiguous())
        kvq.kvq_decode_attention_weights(cfg, x2, q, pool.table_gpu(), pool.lens_gpu(), 200, d ** -0.5, 1.0, w2, o2, ws)
        assert kvq.kvq_read_status(ws) == 0
        assert torch.equal(x1, x2) and torch.equal(o1, o2) and torch.equal(w1, w2)


def test_bad_page_and_overlong_sequence_are_flagged(kvq):
    pool = Pool("int4", 2, 128, [100, 50], 16, 64, 128, seed=5)
    x, q, cfg = pool.gpu(), make_q(2, 4, 128, 9), pool.cfg(kvq)
    table = pool.table_gpu()
    table[0, 2] = pool.num_pages + 7
    w, out = torch.zeros(2, 2, 100, device="cuda"), torch.empty(2, 4, 128, device="cuda")
    ws = kvq.new_weights_workspace(cfg, 2, 4, 100)
    kvq.kvq_decode_attention_weights(cfg, x, q, table, pool.lens_gpu(), 100, 0.1, 1.0, w, out, ws)
    assert kvq.kvq_read_status(ws) == kvq.KVQ_FLAG_BAD_PAGE
    # a length beyond max_len: cut to it and flagged, nothing behind max_len touched
    start = torch.rand(2, 2, 100, device="cuda")
    w = start.clone()
    out, ws = call_weights(kvq, pool, x, q, 1.0, w, max_len=40)
    assert kvq.kvq_read_status(ws) == kvq.KVQ_FLAG_BAD_POSITION
    check_weights(pool, q, 1.0, start, out, w, lens=[40, 40])
    # and one beyond the block table
    lens = torch.tensor([100, 5000], dtype=torch.int32, device="cuda")
    w = start.clone()
    out, ws = call_weights(kvq, pool, x, q, 1.0, w, lens=lens)
    assert kvq.kvq_read_status(ws) & kvq.KVQ_FLAG_BAD_POSITION


def test_int8_half_pages_flag_bad_pages_and_lengths(kvq):
    pool = Pool("int8", 2, 128, [150, 128], 64, 128, 128, seed=5)
    x, q, cfg, table = pool.gpu(), make_q(2, 4, 128, 9), pool.cfg(kvq), pool.table_gpu()
    ws, out = kvq.new_int8_weights_workspace(cfg, 2, 4, 300), torch.empty(2, 4, 128, device="cuda")

    def go(table, lens):
        start = torch.rand(2, 2, 300, device="cuda")
        w = start.clone()
        ws[:4] = 0
        kvq.kvq_int8_decode_attention_weights(cfg, x, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                              300, 128 ** -0.5, 0.0, w, out, ws)
        return start, w, kvq.kvq_read_status(ws)

    for bad in (-1, pool.num_pages):
        t = table.clone()
        t[0, 1] = bad
        assert go(t, [150, 128])[2] == kvq.KVQ_FLAG_BAD_PAGE
    # a length beyond the table's three pages: cut to them and flagged (sequence 1 has two)
    t = table.clone()
    t[1, 2] = t[1, 1]
    start, w, flags = go(t, [150, 200])
    assert flags == kvq.KVQ_FLAG_BAD_POSITION
    assert torch.equal(w[1, :, 192:], start[1, :, 192:])
    # each kv head's weights of 192 positions add up to its two query heads' sums
    assert torch.allclose(w[1, :, :192].double().sum(-1), torch.full((2,), 2.0, dtype=torch.float64, device="cuda"),
                          rtol=1e-4)


# ---- select --------------------------------------------------------------------------------------

def plain_select(w, lens, keep, sinks, recent):
    B, H, _ = w.shape
    kept = np.full((B, H, keep), -1, np.int32)
    for b, n in enumerate(lens):
        for h in range(H):
            x = w[b, h, :n].astype(np.float64)
            x[np.isnan(x)] = -np.inf
            always = np.zeros(n, bool)
            always[:sinks] = True
            always[max(0, n - recent):] = True
            order = np.lexsort((np.arange(n), -x, ~always))
            pick = np.sort(order[:keep])
            kept[b, h, :len(pick)] = pick
    return kept, np.minimum(lens, keep).astype(np.int32)


def run_select(kvq, w, lens, max_len, keep, sinks, recent, status=None):
    B, H, _ = w.shape
    kept = torch.full((B, H, keep), -7, dtype=torch.int32, device="cuda")
    new = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    kvq.kvq_evict_select(kvq.config(H, 128), w, torch.tensor(lens, dtype=torch.int32, device="cuda"), max_len, keep,
                         sinks, recent, kept, new, status=status)
    return kept.cpu().numpy(), new.cpu().numpy()


@pytest.mark.parametrize("lens,keep,sinks,recent", [
    ([1, 0, 2, 5], 1, 0, 0), ([1, 0, 2, 5], 1, 1, 0), ([3, 9, 10, 11], 10, 4, 6), ([100, 7, 64], 64, 4, 16),
    ([1025, 1024, 1023], 511, 0, 1), ([5000, 4097, 33], 33, 1, 31), ([20000, 3], 4096, 4, 512),
    ([70001], 65000, 3, 100), ([131072], 1, 0, 0), ([300, 299], 400, 2, 2), ([32769, 32768, 2048], 9000, 1, 1),
    ([300001], 50000, 7, 1000), ([2049], 2000, 0, 0),
])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd"])
def test_select_matches_numpy(kvq, lens, keep, sinks, recent, kind):
    rng = np.random.default_rng(keep + len(kind))
    B, H, S = len(lens), 3, max(lens) + 3
    w = np.exp(2 * rng.standard_normal((B, H, S))).astype(np.float32)
    if kind == "ties":
        w = np.floor(w)  # many zeros and small whole numbers
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "odd":
        some = rng.integers(0, 12, w.shape)
        for i, v in enumerate((np.nan, np.inf, -np.inf, 0.0, -0.0, -1.5, 1e-42, -1e-42)):
            w[some == i] = v
    got, new = run_select(kvq, torch.from_numpy(w).cuda(), lens, max(lens), keep, sinks, recent)
    want, want_new = plain_select(w, lens, keep, sinks, recent)
    assert np.array_equal(got, want) and np.array_equal(new, want_new)


def test_select_over_long_and_negative_lengths(kvq):
    w = torch.rand(2, 2, 50, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, new = run_select(kvq, w, [60, -4], 40, 8, 1, 2, status=status)
    want, want_new = plain_select(w.cpu().numpy(), [40, 0], 8, 1, 2)
    assert np.array_equal(got, want) and np.array_equal(new, want_new)
    assert status.item() == kvq.KVQ_FLAG_BAD_POSITION


# ---- compact -------------------------------------------------------------------------------------

def random_kept(pool, keep, seed):
    rng = np.random.default_rng(seed)
    kept = np.full((len(pool.lens), pool.Hkv, keep), -1, np.int32)
    for b, n in enumerate(pool.lens):
        for h in range(pool.Hkv):
            m = min(n, keep)
            kept[b, h, :m] = np.sort(rng.permutation(n)[:m])
    return kept


def plain_compact(pool, x, table, dst, kept, w):
    """The pool and weights after the move, row by row from a copy of the pool."""
    y, u = x.copy(), w.copy()
    P = pool.P
    for b, n in enumerate(pool.lens):
        for h in range(pool.Hkv):
            m = min(n, kept.shape[2])
            for i in range(m):
                t = kept[b, h, i]
                for o, rb in zip(pool.off, pool.row):
                    src = x[table[b, t // P], h, o + t % P * rb:o + (t % P + 1) * rb]
                    y[dst[b, i // P], h, o + i % P * rb:o + (i % P + 1) * rb] = src
            u[b, h, :n] = 0
            u[b, h, :m] = w[b, h, kept[b, h, :m]]
    return y, u


def run_compact(kvq, pool, table, dst, kept, w, status=None):
    x, u = pool.gpu(), torch.from_numpy(w.copy()).cuda()
    t = torch.from_numpy(table).cuda()
    fn = kvq.kvq_int8_evict_compact if pool.codec == "int8" else kvq.kvq_evict_compact
    fn(pool.cfg(kvq), x, t, t if dst is table else torch.from_numpy(dst).cuda(), pool.lens_gpu(),
       torch.from_numpy(kept).cuda(), u, status=status)
    return x.cpu().numpy().reshape(pool.bytes.shape), u.cpu().numpy()


@pytest.mark.parametrize("codec,Hkv,d,P,Gk,Gv,lens,keep", [
    ("int4", 4, 128, 16, 64, 128, [600, 0, 1, 77], 64), ("int4", 3, 64, 32, 32, 64, [500, 33], 100),
    ("int4", 1, 64, 16, 64, 64, [1000], 999), ("int4", 2, 256, 64, 128, 32, [700, 64], 65),
    ("int4", 2, 128, 16, 32, 32, [4000], 1500), ("int4", 2, 128, 16, 64, 128, [40, 30], 200),
    ("int8", 2, 128, 64, 128, 128, [300, 5], 77), ("int8", 3, 64, 16, 64, 64, [200], 1),
    ("int8", 2, 256, 32, 128, 128, [3000, 100], 1111),
])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact_moves_rows_bit_for_bit(kvq, codec, Hkv, d, P, Gk, Gv, lens, keep, in_place):
    blocks = (keep + P - 1) // P
    pool = Pool(codec, Hkv, d, lens, P, Gk, Gv, seed=keep, spare=1 if in_place else len(lens) * blocks)
    dst = pool.table if in_place else pool.spare[:len(lens) * blocks].reshape(len(lens), blocks).copy()
    kept = random_kept(pool, keep, 3)
    w = np.random.default_rng(1).random((len(lens), Hkv, max(lens) + 2)).astype(np.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, u = run_compact(kvq, pool, pool.table, dst, kept, w, status)
    want_x, want_u = plain_compact(pool, pool.bytes, pool.table, dst, kept, w)
    assert status.item() == 0
    assert np.array_equal(x, want_x) and np.array_equal(u, want_u)


def test_compact_skips_and_flags_bad_positions_and_pages(kvq):
    pool = Pool("int4", 2, 128, [100, 90], 16, 64, 128, seed=4)
    kept = random_kept(pool, 40, 8)
    w = np.random.default_rng(1).random((2, 2, 100)).astype(np.float32)
    bad = kept.copy()
    bad[0, 1, 39] = 100  # outside the sequence
    bad[1, 0, 0] = -3
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, _ = run_compact(kvq, pool, pool.table, pool.table, bad, w, status)
    assert status.item() == kvq.KVQ_FLAG_BAD_POSITION
    want, _ = plain_compact(pool, pool.bytes, pool.table, pool.table, kept, w)
    ours = pool.table[0, :3], pool.table[1, :3]
    for b, h, rows in ((0, 0, 40), (0, 1, 39), (1, 1, 40)):
        for i in range(rows):
            at = (ours[b][i // 16], h, i % 16)
            assert pool.stored(x, *at) == pool.stored(want, *at)
    # a bad source page and a bad destination page
    status.zero_()
    table = pool.table.copy()
    table[0, 0] = -1
    x, _ = run_compact(kvq, pool, table, table, kept, w, status)
    assert status.item() == kvq.KVQ_FLAG_BAD_PAGE
    untouched = np.setdiff1d(np.arange(pool.num_pages), np.concatenate([table[0, :3], table[1, :3]]))
    assert np.array_equal(x[untouched], pool.bytes[untouched])
    # a destination table that is too short for the rows kept
    status.zero_()
    x, _ = run_compact(kvq, pool, pool.table, np.ascontiguousarray(pool.table[:, :2]), kept, w, status)
    assert status.item() == kvq.KVQ_FLAG_BAD_POSITION


def test_compact_without_weights(kvq):
    pool = Pool("int4", 2, 128, [100], 16, 64, 128, seed=4)
    kept = random_kept(pool, 30, 8)
    x, table = pool.gpu(), pool.table_gpu()
    kvq.kvq_evict_compact(pool.cfg(kvq), x, table, table, pool.lens_gpu(), torch.from_numpy(kept).cuda())
    want, _ = plain_compact(pool, pool.bytes, pool.table, pool.table, kept, np.zeros((1, 2, 100), np.float32))
    assert np.array_equal(x.cpu().numpy().reshape(want.shape), want)


# ---- together ------------------------------------------------------------------------------------

def test_serving_loop_with_eviction(kvq):
    """Append a history, decode with tracked weights, cut the cache, decode on: after the cut each KV head attends to
    exactly the positions it kept, and the next tokens follow behind them."""
    from int4_group_quantized_kvq_gb300.cache import PagedKVCache
    B, H, r, d, P, n0 = 2, 3, 2, 128, 16, [150, 90]
    blocks = 16
    cfg = kvq.config(H, d, P, 64, 128, B * blocks)
    table = torch.randperm(B * blocks, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, blocks)
    cache = PagedKVCache(cfg, table, H * r, blocks * P, track_weights=True, decay=0.9)
    gen = torch.Generator(device="cuda").manual_seed(5)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda").half()

    for b in range(B):  # histories of different lengths
        one = PagedKVCache(cfg, cache.block_table[b:b + 1], H * r, blocks * P, pool=cache.pool)
        one.append(rand(1, n0[b], H, d), rand(1, n0[b], H, d), torch.zeros(1, dtype=torch.int32, device="cuda"))
    lens = torch.tensor(n0, dtype=torch.int32, device="cuda")
    out = torch.empty(B, H * r, d, device="cuda")

    def step():
        nonlocal lens
        q, k, v = rand(B, H * r, d), rand(B, H, d), rand(B, H, d)
        lens = lens + 1
        cache.decode_step(q, k, v, lens - 1, lens, out)
        return q

    def rows(b, n):
        k, v = torch.empty(n, H, d, device="cuda"), torch.empty(n, H, d, device="cuda")
        kvq.kvq_dequantize(cfg, cache.pool, cache.block_table, b, 0, n, k, v)
        return k.double().cpu().numpy().transpose(1, 0, 2), v.double().cpu().numpy().transpose(1, 0, 2)

    for _ in range(5):
        step()
    keep, sinks, recent = 100, 4, 20
    weights = cache.weights.cpu().numpy()
    old = [rows(b, n0[b] + 5) for b in range(B)]
    lens = cache.evict(lens, keep, sinks, recent)
    assert lens.tolist() == [100, 95] and cache.flags() == 0
    kept, _ = plain_select(weights, [n0[0] + 5, n0[1] + 5], keep, sinks, recent)
    for b in range(B):
        m = int(lens[b])
        k, v = rows(b, m)
        for h in range(H):
            at = kept[b, h, :m]
            assert np.array_equal(k[h], old[b][0][h][at]) and np.array_equal(v[h], old[b][1][h][at])
            assert np.array_equal(cache.weights[b, h, :m].cpu().numpy(), weights[b, h, at])
            assert not cache.weights[b, h, m:].any()
    q = step()
    for b in range(B):
        K, V = rows(b, int(lens[b]))
        for hq in range(H * r):
            z = q[b, hq].double().cpu().numpy() @ K[hq // r].T * d ** -0.5
            dz = score_error(q[b, hq:hq + 1].double().cpu().numpy(), K[hq // r], d ** -0.5)
            tol, _ = errors(z, V[hq // r], dz)
            assert np.abs(out[b, hq].cpu().numpy() - softmax64(z) @ V[hq // r]).max() <= tol
    # a second cut, into other pages
    other = torch.arange(B * blocks, dtype=torch.int32, device="cuda")
    used = torch.cat([cache.block_table[b, :(int(lens[b]) + P - 1) // P] for b in range(B)])
    spare = other[~torch.isin(other, used)][:B * 4].view(B, 4).contiguous()
    before = [rows(b, int(lens[b])) for b in range(B)]
    weights = cache.weights.cpu().numpy()
    old_lens = lens.tolist()
    lens = cache.evict(lens, 60, 4, 20, dst_table=spare)
    kept, _ = plain_select(weights, old_lens, 60, 4, 20)
    assert lens.tolist() == [60, 60] and cache.flags() == 0
    for b in range(B):
        k, v = rows(b, 60)
        for h in range(H):
            assert np.array_equal(k[h], before[b][0][h][kept[b, h]]) and np.array_equal(v[h], before[b][1][h][kept[b, h]])


def test_decode_right_behind_select_and_compact(kvq):
    """Decode attention launched directly behind the two kernels reads the lengths and rows that they wrote."""
    pool = Pool("int4", 2, 128, [3000, 2500], 16, 64, 128, seed=6)
    cfg, q = pool.cfg(kvq), make_q(2, 8, 128, 2)
    w = torch.rand(2, 2, 3000, device="cuda")
    kept = torch.empty(2, 2, 700, dtype=torch.int32, device="cuda")
    ws, table, lens = kvq.new_workspace(cfg, 2, 8, 3000), pool.table_gpu(), pool.lens_gpu()

    def go(wait):
        x, new = pool.gpu(), torch.full((2,), 3000, dtype=torch.int32, device="cuda")
        out, u = torch.zeros(2, 8, 128, device="cuda"), w.clone()
        torch.cuda.synchronize()
        kvq.kvq_evict_select(cfg, u, lens, 3000, 700, 4, 64, kept, new)
        if wait:
            torch.cuda.synchronize()
        kvq.kvq_evict_compact(cfg, x, table, table, lens, kept, u)
        if wait:
            torch.cuda.synchronize()
        kvq.kvq_decode_attention(cfg, x, q, table, new, 3000, 128 ** -0.5, out, ws)
        return out.clone()

    want = go(True)
    for _ in range(5):
        assert torch.equal(go(False), want)


def test_nothing_to_attend_and_no_positions(kvq):
    pool = Pool("int4", 2, 128, [0, 0], 16, 64, 128, seed=6)
    cfg, q = pool.cfg(kvq), make_q(2, 4, 128, 2)
    w, out = torch.full((2, 2, 9), 3.0, device="cuda"), torch.full((2, 4, 128), 7.0, device="cuda")
    ws = kvq.new_weights_workspace(cfg, 2, 4, 9)
    kvq.kvq_decode_attention_weights(cfg, pool.gpu(), q, pool.table_gpu(), pool.lens_gpu(), 9, 0.1, 1.0, w, out, ws)
    assert not out.any() and (w == 3.0).all() and kvq.kvq_read_status(ws) == 0
    none = torch.empty(2, 2, 0, device="cuda")
    kvq.kvq_decode_attention_weights(cfg, pool.gpu(), q, pool.table_gpu(), pool.lens_gpu(), 0, 0.1, 1.0, none, out, ws)
    got, new = run_select(kvq, none, [0, 0], 0, 3, 1, 1)
    assert (got == -1).all() and not new.any()
    x, u = run_compact(kvq, pool, pool.table, pool.table, got, np.zeros((2, 2, 4), np.float32))
    assert np.array_equal(x, pool.bytes) and not u.any()


def test_a_row_of_nan_stays_in_its_row(kvq):
    for Hkv, r in ((8, 1), (2, 4)):
        pool = Pool("int4", Hkv, 128, [70, 90], 16, 64, 128, seed=6)
        q = make_q(2, Hkv * r, 128, 2)
        clean, w0 = q.clone(), torch.zeros(2, Hkv, 90, device="cuda")
        out0, _ = call_weights(kvq, pool, pool.gpu(), clean, 1.0, w0)
        q[0, 1, 5] = float("nan")
        w1 = torch.zeros(2, Hkv, 90, device="cuda")
        out1, _ = call_weights(kvq, pool, pool.gpu(), q, 1.0, w1)
        rows = torch.ones(2, Hkv * r, dtype=torch.bool)
        rows[0, 1] = False
        heads = torch.ones(2, Hkv, dtype=torch.bool)
        heads[0, 1 // r] = False
        assert torch.equal(out0.cpu()[rows], out1.cpu()[rows]) and torch.equal(w0.cpu()[heads], w1.cpu()[heads])


def test_select_and_compact_replayed_from_a_graph(kvq):
    pool = Pool("int8", 2, 128, [3000, 40], 32, 128, 128, seed=6)
    cfg, table, lens = pool.cfg(kvq), pool.table_gpu(), pool.lens_gpu()
    x, w = pool.gpu(), torch.rand(2, 2, 3000, device="cuda")
    x0, w0 = x.clone(), w.clone()
    kept, new = torch.empty(2, 2, 500, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")

    def go():
        kvq.kvq_evict_select(cfg, w, lens, 3000, 500, 4, 64, kept, new)
        kvq.kvq_int8_evict_compact(cfg, x, table, table, lens, kept, w)

    go()
    want = x.clone(), w.clone(), kept.clone(), new.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(2):
        x.copy_(x0)
        w.copy_(w0)
        kept.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, (x, w, kept, new)))


@pytest.mark.parametrize("as_handle", [False, True])
def test_evict_on_a_side_stream(kvq, as_handle):
    from int4_group_quantized_kvq_gb300.cache import PagedKVCache
    pool = Pool("int4", 2, 128, [200, 90], 16, 64, 128, seed=4)
    w = torch.rand(2, 2, 200, device="cuda")
    caches = [PagedKVCache(pool.cfg(kvq), pool.table_gpu(), 4, 200, pool=pool.gpu(), track_weights=True) for _ in range(2)]
    for c in caches:
        c.weights.copy_(w)
    want = caches[0].evict(pool.lens_gpu(), 50, 2, 8)
    side, lens = torch.cuda.Stream(), pool.lens_gpu()
    side.wait_stream(torch.cuda.current_stream())
    got = caches[1].evict(lens, 50, 2, 8, stream=side.cuda_stream if as_handle else side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(caches[0].pool, caches[1].pool)
    assert torch.equal(caches[0].weights, caches[1].weights)


def test_cache_refuses_what_it_does_not_track(kvq):
    from int4_group_quantized_kvq_gb300.cache import HostPipeline, HostStaging, PagedKVCache
    cfg = kvq.config(2, 128, 16, 64, 128, 8)
    table = torch.arange(8, dtype=torch.int32).view(1, 8)
    lens = torch.tensor([20], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        PagedKVCache(cfg, table, 4, 128, window=16, track_weights=True)
    plain, tracked = PagedKVCache(cfg, table, 4, 128), PagedKVCache(cfg, table, 4, 128, track_weights=True)
    with pytest.raises(ValueError):
        plain.evict(lens, 10)
    with pytest.raises(ValueError):
        plain.attend_diff(None, None, lens, None)
    with pytest.raises(ValueError):
        tracked.evict(lens, 100, dst_table=table[:, :2].cuda().contiguous())
    with pytest.raises(ValueError):
        tracked.decode_step_host(HostStaging(1, 4, 2, 128, "cuda"), lens, lens)
    with pytest.raises(ValueError):
        HostPipeline(tracked).step(0, lens, lens)


def test_tensors_are_checked(kvq):
    pool = Pool("int4", 2, 128, [100, 50], 16, 64, 128, seed=5)
    x, q, cfg = pool.gpu(), make_q(2, 4, 128, 9), pool.cfg(kvq)
    table, lens = pool.table_gpu(), pool.lens_gpu()
    w, out = torch.zeros(2, 2, 100, device="cuda"), torch.empty(2, 4, 128, device="cuda")
    ws = kvq.new_weights_workspace(cfg, 2, 4, 100)

    def call(**k):
        a = dict(cfg=cfg, pool=x, q=q, block_table=table, seq_lens=lens, max_len=100, softmax_scale=0.1, decay=1.0,
                 weights=w, out=out, workspace=ws)
        a.update(k)
        kvq.kvq_decode_attention_weights(**a)

    call()
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=q.cpu()), dict(pool=x[:-1]), dict(block_table=table[:1]),
                dict(seq_lens=lens.long()), dict(seq_lens=lens[:1]), dict(weights=w[:, :1].contiguous()),
                dict(weights=w.transpose(0, 1)), dict(weights=w.double()), dict(out=out[:1]), dict(out=None),
                dict(weights=w[:, :, ::2])):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(decay=1.5), dict(decay=float("nan")), dict(max_len=101), dict(max_len=-1),
                dict(workspace=ws[:256].clone())):
        with pytest.raises(kvq.KvqError):
            call(**bad)
    kept, new = torch.empty(2, 2, 10, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    for bad in (dict(kept=kept[:1]), dict(kept=kept.long()), dict(new_lens=new[:1]), dict(weights=w[:1]),
                dict(status=torch.zeros(1))):
        a = dict(cfg=cfg, weights=w, seq_lens=lens, max_len=100, keep=10, sinks=1, recent=1, kept=kept, new_lens=new)
        a.update(bad)
        with pytest.raises(ValueError):
            kvq.kvq_evict_select(**a)
    with pytest.raises(ValueError):
        kvq.kvq_evict_compact(cfg, x, table, table, lens, kept[:1].contiguous(), w)
    with pytest.raises(ValueError):
        kvq.kvq_evict_compact(cfg, x, table, table[:1].contiguous(), lens, kept, w)


@pytest.mark.parametrize("form", ["weights", "int8 weights", "differential", "plain"])
def test_block_table_of_more_than_31_bits_of_positions(kvq, form):
    """A table of 2^25 pages of 64 tokens: what a short table of the same pages gives."""
    codec = "int8" if form == "int8 weights" else "int4"
    pool = Pool(codec, 2, 128, [150], 64, 64, 128, seed=13)
    x, q, cfg, lens = pool.gpu(), make_q(1, 8, 128, 14), pool.cfg(kvq), pool.lens_gpu()
    short = pool.table_gpu()
    long = torch.full((1, 1 << 25), -1, dtype=torch.int32, device="cuda")
    long[:, :short.shape[1]] = short
    lam = torch.full((8,), 0.4, device="cuda")

    def go(table):
        w, out = torch.rand(1, 2, 150, generator=torch.Generator("cuda").manual_seed(1), device="cuda"), \
            torch.zeros(1, 8, 128, device="cuda")
        args = cfg, x, q, table, lens, 150, 0.1
        if form == "plain":
            ws = kvq.new_workspace(cfg, 1, 8, 150)
            kvq.kvq_decode_attention(*args, out, ws)
        elif form == "differential":
            ws = kvq.new_diff_workspace(cfg, 1, 8, 150)
            kvq.kvq_diff_decode_attention(*args, lam, None, 0.0, 1.0, out, ws)
        elif codec == "int8":
            ws = kvq.new_int8_weights_workspace(cfg, 1, 8, 150)
            kvq.kvq_int8_decode_attention_weights(*args, 1.0, w, out, ws)
        else:
            ws = kvq.new_weights_workspace(cfg, 1, 8, 150)
            kvq.kvq_decode_attention_weights(*args, 1.0, w, out, ws)
        assert kvq.kvq_read_status(ws) == 0
        return w, out

    (w0, o0), (w1, o1) = go(short), go(long)
    assert o0.any() and torch.equal(w0, w1) and torch.equal(o0, o1)


def test_a_row_that_is_not_moved_has_weight_zero(kvq):
    pool = Pool("int4", 2, 128, [100, 90], 16, 64, 128, seed=4)
    kept = random_kept(pool, 40, 8)
    w = 1 + np.random.default_rng(1).random((2, 2, 100)).astype(np.float32)
    _, want = plain_compact(pool, pool.bytes, pool.table, pool.table, kept, w)
    # positions outside the sequence
    bad, expect = kept.copy(), want.copy()
    bad[0, 1, 39], expect[0, 1, 39] = 100, 0
    bad[1, 0, 0], expect[1, 0, 0] = -3, 0
    _, u = run_compact(kvq, pool, pool.table, pool.table, bad, w)
    assert np.array_equal(u, expect)
    # pages out of range: a source's (in place also a destination's), and a destination's alone
    table = pool.table.copy()
    table[0, 1] = pool.num_pages
    _, u = run_compact(kvq, pool, table, table, kept, w)
    expect = want.copy()
    for h in range(2):
        for i in range(40):
            if kept[0, h, i] // 16 == 1 or i // 16 == 1:
                expect[0, h, i] = 0
    assert np.array_equal(u, expect) and (expect != want).any()
    _, u = run_compact(kvq, pool, pool.table, table, kept, w)
    expect = want.copy()
    expect[0, :, 16:32] = 0
    assert np.array_equal(u, expect)
    # positions behind a short destination table
    _, u = run_compact(kvq, pool, pool.table, np.ascontiguousarray(pool.table[:, :2]), kept, w)
    expect = want.copy()
    expect[:, :, 32:40] = 0
    assert np.array_equal(u, expect)


def test_evict_in_place_asks_for_no_more_pages_than_the_cache_has(kvq):
    from int4_group_quantized_kvq_gb300.cache import PagedKVCache
    pool = Pool("int4", 2, 128, [100, 60], 16, 64, 128, seed=4)  # 7 pages a sequence: 112 positions
    cache = PagedKVCache(pool.cfg(kvq), pool.table_gpu(), 4, 200, pool=pool.gpu(), track_weights=True)
    cache.weights.copy_(torch.rand(2, 2, 200, device="cuda"))
    w = cache.weights.clone()
    assert cache.evict(pool.lens_gpu(), 150, 2, 8).tolist() == [100, 60]
    assert cache.flags() == 0
    assert np.array_equal(cache.pool.cpu().numpy().reshape(pool.bytes.shape), pool.bytes)
    assert torch.equal(cache.weights[0, :, :100], w[0, :, :100]) and torch.equal(cache.weights[1, :, :60], w[1, :, :60])
    with pytest.raises(ValueError):  # 112 positions do not fit into 6 pages
        cache.evict(pool.lens_gpu(), 150, 2, 8, dst_table=cache.block_table[:, :6].contiguous())


@pytest.mark.parametrize("current", [False, True])
def test_evict_on_a_side_stream_holds_the_table_it_reads(kvq, current):
    """The old block table's memory is not handed out while the side stream may still read it."""
    from int4_group_quantized_kvq_gb300.cache import PagedKVCache
    pool = Pool("int4", 2, 128, [200], 16, 64, 128, seed=4, spare=8)
    wide = np.full((1, 1 << 20), -1, np.int32)  # 4 MB, found again by the next requests of its size
    wide[:, :pool.blocks] = pool.table
    cache = PagedKVCache(pool.cfg(kvq), torch.from_numpy(wide), 4, 200, pool=pool.gpu(), track_weights=True)
    cache.weights.copy_(torch.rand(1, 2, 200, device="cuda"))
    dst, lens = torch.from_numpy(pool.spare[:4][None].copy()).cuda(), pool.lens_gpu()
    first = cache.block_table.data_ptr()
    last = first + 4 * wide.size
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    if current:
        with torch.cuda.stream(side):
            cache.evict(lens, 60, 2, 8, dst_table=dst)
    else:
        cache.evict(lens, 60, 2, 8, dst_table=dst, stream=side)
    assert not side.query(), "the side stream is still busy"
    new = [torch.empty(1 << 20, dtype=torch.int32, device="cuda") for _ in range(16)]
    assert all(t.data_ptr() + 4 * t.numel() <= first or t.data_ptr() >= last for t in new)
    side.synchronize()
    assert cache.flags() == 0


# Calls that leave the weights to a kernel of their own: more than 152 rows of the output and chunks of weights.
@pytest.mark.parametrize("codec,Hkv,r,d,P,Gk,Gv,lens", [
    ("int4", 32, 1, 128, 16, 64, 128, [300, 31, 0, 513, 17]),            # four kv heads a unit
    ("int4", 32, 1, 128, 16, 64, 128, [(37 * b) % 200 for b in range(20)]),  # 640 rows: the light combine
    ("int4", 7, 1, 128, 64, 32, 64, [64, 63, 1, 700] * 6),
    ("int4", 16, 2, 128, 16, 32, 32, [2049, 5, 100, 16, 0]),             # two kv heads a unit
    ("int4", 8, 5, 128, 16, 64, 128, [300, 31, 1, 700]),                 # two slots a thread
    ("int4", 4, 8, 128, 32, 128, 64, [999, 64, 65, 1, 0]),
    ("int4", 4, 4, 128, 16, 64, 128, [40001]),                           # rows of many partials, many chunks
    ("int4", 8, 7, 64, 32, 64, 32, [400, 255, 1]),
    ("int4", 16, 4, 256, 16, 64, 128, [300, 17, 129]),
    ("int4", 33, 1, 256, 64, 128, 32, [129, 0, 640, 1, 2]),
    ("int8", 8, 5, 128, 64, 128, 128, [300, 1291, 701, 65, 33]),         # half-page units, two slots a thread
    ("int8", 4, 8, 128, 16, 128, 128, [513, 40, 1, 0, 200]),
    ("int8", 40, 1, 128, 32, 128, 128, [33, 250, 64, 1]),
])
@pytest.mark.parametrize("decay", [1.0, 0.0, 0.75])
def test_weights_in_a_launch_of_their_own_match_fp64(kvq, codec, Hkv, r, d, P, Gk, Gv, lens, decay):
    chunk = 256 * (8 if r == 1 else 16 // (2 if r == 2 else 4 if r <= 4 else 8))
    assert len(lens) * Hkv * (r + -(-max(lens) // chunk)) > 152
    pool = Pool(codec, Hkv, d, lens, P, Gk, Gv, seed=d + r, poison=True)
    q = make_q(len(lens), Hkv * r, d, 3)
    before = torch.rand(len(lens), Hkv, max(lens) + 5, device="cuda")
    if decay == 0.0:
        before.fill_(float("nan"))  # not read
    weights = before.clone()
    out, ws = call_weights(kvq, pool, pool.gpu(), q, decay, weights)
    assert kvq.kvq_read_status(ws) == 0
    check_weights(pool, q, decay, before, out, weights)
