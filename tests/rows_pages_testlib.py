"""Pools made row by row for the tests of attention's precision: few kinds of pages, named as often as wanted by a block
table, over one kv head of the INT4 cache or a latent cache."""
from __future__ import annotations

import numpy as np
import torch


def nibbles(codes):
    n = (np.asarray(codes) + 8).astype(np.uint8)
    return n[0::2] | n[1::2] << 4


def halves(x):
    return np.asarray(x, np.float16).view(np.uint8)


class Kv:
    """INT4 cache of one kv head; a row is (key codes, key scales, value codes, value scales)."""

    def __init__(self, d=64, r=1, P=64, G=32, rows=1):
        self.d, self.heads, self.P, self.G, self.rows, self.latent = d, r, P, G, rows, False

    def page(self, rows):
        parts = [np.concatenate([f(row[i]) for row in rows]) for i, f in ((0, nibbles), (2, nibbles), (1, halves), (3, halves))]
        x = np.concatenate(parts)
        return np.pad(x, (0, -len(x) % 16))

    def row(self, kv):
        """A row from (codes, scales) of the key and of the value; an int for a vector of it."""
        return tuple(np.full(self.d if i % 2 == 0 else self.d // self.G, x) if np.isscalar(x) else np.asarray(x)
                     for i, x in enumerate(kv))

    def values(self, row):
        """fp64 key and value of a row."""
        return [row[i].astype(np.float64) * np.repeat(row[i + 1].astype(np.float16).astype(np.float64), self.G) for i in (0, 2)]

    def run(self, kvq, pages, table, lens, new, q, scale):
        """q fp16 [heads, d], the same for every row; the outputs, fp64 [rows, heads, d]."""
        pool = torch.from_numpy(np.concatenate([self.page(x) for x in pages])).cuda()
        cfg = kvq.config(1, self.d, self.P, self.G, self.G, len(pages))
        return attend(kvq, kvq.kvq_chunk_attention, kvq.new_chunk_workspace, cfg, pool, table, lens, new, q, scale, self.d)


class Latents:
    """Latent cache; a row is (codes, scales, rotary key)."""

    def __init__(self, L=256, heads=1, P=64, G=64, rows=1):
        self.d, self.heads, self.P, self.G, self.rows, self.latent = L, heads, P, G, rows, True

    def page(self, rows):
        return np.concatenate([np.concatenate([f(row[i]) for row in rows]) for i, f in ((0, nibbles), (1, halves), (2, halves))])

    def run(self, kvq, pages, table, lens, new, q, scale):
        pool = torch.from_numpy(np.concatenate([self.page(x) for x in pages])).cuda()
        cfg = kvq.latent_config(self.d, 64, self.P, self.G, len(pages))
        q = np.concatenate([q, np.zeros((len(q), 64))], axis=-1) if q.shape[-1] == self.d else q
        return attend(kvq, kvq.kvq_latent_attention, kvq.new_latent_workspace, cfg, pool, table, lens, new, q, scale, self.d)


def attend(kvq, fn, new_workspace, cfg, pool, table, lens, new, q, scale, width):
    def ints(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    cu = np.concatenate([[0], np.cumsum(new)])
    gq = torch.from_numpy(np.tile(q.astype(np.float16), (int(cu[-1]), 1, 1))).cuda()
    out = torch.full((int(cu[-1]), len(q), width), 7.0, dtype=torch.float16, device="cuda")
    ws = new_workspace(cfg, len(new), len(q), int(max(lens)))
    fn(cfg, pool, gq, ints(table), ints(lens), ints(cu), int(max(lens)), scale, out, ws)
    assert kvq.kvq_read_status(ws) == 0
    return out.cpu().numpy().astype(np.float64)
