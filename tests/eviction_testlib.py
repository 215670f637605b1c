"""Shared by the eviction and differential-attention tests: pools of random rows, their values read byte by byte
in numpy, and attention in fp64 over them."""
from __future__ import annotations

import numpy as np
import torch

EPS32 = 2.0 ** -24  # half a step of fp32


class Pool:
    """A random pool of `codec` ("int4" or "int8") with a block table for sequences of `lens` positions.

    Rows hold random codes over the whole code range and scales of a few binades, as the quantizers store them;
    with `poison` every byte that no position owns is 0xFF, a NaN as a scale."""

    def __init__(self, codec, Hkv, d, lens, P=16, Gk=64, Gv=64, seed=0, spare=2, blocks=None,
                 poison=False):
        self.codec, self.Hkv, self.d, self.P, self.Gk, self.Gv, self.lens = codec, Hkv, d, P, Gk, Gv, list(lens)
        rng = np.random.default_rng(seed)
        pages = [(n + P - 1) // P for n in self.lens]
        self.blocks = max(1, max(pages)) if blocks is None else blocks
        self.num_pages = sum(pages) + spare
        order = rng.permutation(self.num_pages)
        self.table = np.full((len(self.lens), self.blocks), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.spare = order[at:].astype(np.int32)
        self.row = (d, d, 4, 4) if codec == "int8" else (d // 2, d // 2, 2 * (d // Gk), 2 * (d // Gv))
        self.off = [P * sum(self.row[:i]) for i in range(4)]
        self.block = (P * sum(self.row) + 15) // 16 * 16
        x = np.zeros((self.num_pages, Hkv, self.block), np.uint8)
        for i in range(4):
            shape = (self.num_pages, Hkv, P * self.row[i])
            if i < 2:
                if codec == "int8":
                    v = rng.integers(-127, 128, shape).astype(np.int8).view(np.uint8)
                else:
                    v = (rng.integers(1, 16, shape) | rng.integers(1, 16, shape) << 4).astype(np.uint8)
            else:
                base = 0.02 if codec == "int8" else 0.3
                n = P * self.row[i] // (4 if codec == "int8" else 2)
                s = base * np.exp2(rng.uniform(-2, 1, (self.num_pages, Hkv, n)))
                v = s.astype(np.float32 if codec == "int8" else np.float16).view(np.uint8)
            x[:, :, self.off[i]:self.off[i] + v.shape[-1]] = v
        if poison:  # slots behind each sequence's end, and spare pages: NaN scales and extreme codes
            x[self.spare] = 0xFF
            for b, n in enumerate(self.lens):
                for slot in range(n % P if n else 0, P if n % P else 0):
                    for o, r in zip(self.off, self.row):
                        x[self.table[b, n // P], :, o + slot * r:o + (slot + 1) * r] = 0xFF
        self.bytes = x

    def cfg(self, kvq):
        return kvq.config(self.Hkv, self.d, self.P, self.Gk, self.Gv, self.num_pages)

    def gpu(self):
        return torch.from_numpy(self.bytes.reshape(-1).copy()).cuda()

    def table_gpu(self):
        return torch.from_numpy(self.table).cuda()

    def lens_gpu(self):
        return torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def stored(self, x, page, h, slot):
        """The four stored pieces of a token row, as bytes; x the pool [num_pages, Hkv, block]."""
        return [x[page, h, o + slot * r:o + (slot + 1) * r].tobytes() for o, r in zip(self.off, self.row)]

    def values(self, b, n, x=None, table=None):
        """fp64 K and V [Hkv, n, d] of sequence b's first n positions."""
        x = self.bytes if x is None else x
        table = self.table if table is None else table
        out = []
        t = np.arange(n)
        page = table[b, t // self.P]
        for part, group in ((0, self.Gk), (1, self.Gv)):
            def piece(i):
                at = self.off[i] + (t % self.P)[:, None] * self.row[i] + np.arange(self.row[i])
                return np.stack([x[page[:, None], h, at] for h in range(self.Hkv)])  # [H, n, bytes]
            c, s = piece(part), np.ascontiguousarray(piece(2 + part))
            if self.codec == "int8":
                out.append(c.view(np.int8).astype(np.float64) * s.view(np.float32).astype(np.float64))
                continue
            codes = np.stack([c & 15, c >> 4], axis=-1).reshape(*c.shape[:2], self.d).astype(np.float64) - 8
            out.append(codes * np.repeat(s.view(np.float16).astype(np.float64), group, axis=-1))
        return out


def softmax64(z):
    e = np.exp(z - z.max(axis=-1, keepdims=True))
    return e / e.sum(axis=-1, keepdims=True)


def score_error(q, K, scale):
    """A bound on |computed - exact score| of any (query, position), in natural-log units.

    Products of codes and q are exact in fp32.  A k-step of the MMA adds 16 products and the running sum with at most
    one truncated ulp (2 EPS32) of the largest intermediate each way, d / 16 of them; the group scales, the softmax
    scale (two roundings) and the running sum over groups add a handful of EPS32 more; all relative to sum |q k|."""
    d = K.shape[-1]
    mag = np.abs(q) @ np.abs(K).T * scale
    return (2 * (d / 16) + 8) * EPS32 * mag.max()


def errors(z, V, dz, codec="int4"):
    """Bounds (output, absolute per element; softmax weight, relative) for one query row's exact scores z [n] known to
    dz and its values V [n, d]:
      scores         2 dz relative to each weight (numerator and sum);
      exp2           its argument z log2 e - max, three roundings; the hardware's 2^-22, once per position and once
                     per partial (rescalings multiply numerator and sum alike);
      f16 hi + lo    2^-22 relative; an absolute 2^-25 where the low part is subnormal, on terms of up to 2^kUp (2 for
                     INT4, 6 for INT8) times a code of at most 7 (127), against the sum l of the terms;
      fp32 sums      one truncated ulp for each 16-position step of the MMA, a few for the merge of the partials."""
    n = len(z)
    top = np.abs(z).max()
    rel = 2 * dz + 3 * EPS32 * (2 * top + 2) + 2 * 2.0 ** -22 + 8 * EPS32
    l = np.exp(z - z.max()).sum()
    code, up = (127, 64) if codec == "int8" else (7, 4)
    sub = n * 2.0 ** -25 * code / (up * l)
    vmax = np.abs(V).max()
    return (rel + 2.0 ** -22 + 2 * EPS32 * (n / 16 + 16)) * vmax + sub, rel + 2 * EPS32 * (n / 32 + 16)
