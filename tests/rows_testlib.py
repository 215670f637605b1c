"""Shared by the tests of the calls on ragged batches of rows: latent pools, rotary positions in numpy, attention
of many rows in fp64 and the bounds of its fp16 form."""
from __future__ import annotations

import numpy as np
import torch

from eviction_testlib import softmax64

HALF_STEP = 2.0 ** -11  # a rounding to fp16 is off by at most this, relative (half a step)
EPS32 = 2.0 ** -24


class LatentPool:
    """A random latent pool with a block table for sequences of `lens` positions; with `poison` every byte that no
    position owns is 0xFF (NaN scales and rotary keys)."""

    def __init__(self, L, lens, P=64, G=64, seed=0, spare=2, poison=True, R=64):
        self.L, self.R, self.P, self.G, self.lens = L, R, P, G, list(lens)
        rng = np.random.default_rng(seed)
        pages = [(n + P - 1) // P for n in lens]
        self.blocks = max(1, max(pages))
        self.num_pages = sum(pages) + spare
        order = rng.permutation(self.num_pages)
        self.table = np.full((len(lens), self.blocks), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.row = (L // 2, 2 * (L // G), 2 * R)
        self.off = [P * sum(self.row[:i]) for i in range(3)]
        x = np.zeros((self.num_pages, P * sum(self.row)), np.uint8)
        shape = (self.num_pages, P * L // 2)
        x[:, :self.off[1]] = rng.integers(1, 16, shape) | rng.integers(1, 16, shape) << 4
        s = (0.3 * np.exp2(rng.uniform(-2, 1, (self.num_pages, P * (L // G))))).astype(np.float16)
        x[:, self.off[1]:self.off[2]] = s.view(np.uint8)
        x[:, self.off[2]:] = rng.standard_normal((self.num_pages, P * R)).astype(np.float16).view(np.uint8)
        if poison:
            x[order[at:]] = 0xFF
            for b, n in enumerate(self.lens):
                for slot in range(n % P, P if n % P else 0):
                    for o, r in zip(self.off, self.row):
                        x[self.table[b, n // P], o + slot * r:o + (slot + 1) * r] = 0xFF
        self.bytes = x

    def cfg(self, kvq):
        return kvq.latent_config(self.L, self.R, self.P, self.G, self.num_pages)

    def gpu(self):
        return torch.from_numpy(self.bytes.reshape(-1).copy()).cuda()

    def table_gpu(self):
        return torch.from_numpy(self.table).cuda()

    def rows(self, b, n, x=None):
        """fp64 [n, L + R]: sequence b's first n rows."""
        x = self.bytes if x is None else x.reshape(self.num_pages, -1)
        t = np.arange(n)
        page = self.table[b, t // self.P][:, None]

        def piece(i):
            return np.ascontiguousarray(x[page, self.off[i] + (t % self.P)[:, None] * self.row[i] + np.arange(self.row[i])])

        c = piece(0)
        codes = np.stack([c & 15, c >> 4], axis=-1).reshape(n, self.L).astype(np.float64) - 8
        lat = codes * np.repeat(piece(1).view(np.float16).astype(np.float64), self.G, axis=-1)
        return np.concatenate([lat, piece(2).view(np.float16).astype(np.float64)], axis=-1)


def ragged(new, pad=0):
    """cu_rows of these row counts, and the rows of the arrays with `pad` behind them."""
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return cu, int(cu[-1]) + pad


def angles(length, rot):
    """fp32 [length, rot]: cosines, then sines."""
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(length)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], axis=-1).astype(np.float32)


def turned(x, cs, rot, inter):
    """fp16 x [rows, heads, d], its first rot elements turned by cs [rows, rot]: fp32, each operation rounded once."""
    y = x.astype(np.float32)
    c, n = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    i = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
    j = i + 1 if inter else i + rot // 2
    a, b = y[..., i].copy(), y[..., j].copy()
    y[..., i] = a * c - b * n
    y[..., j] = b * c + a * n
    return y.astype(np.float16)


def attend64(q, K, V, first, scale):
    """fp64 q [rows, n] at positions first, first + 1, ..: (outputs [rows, m], bounds [rows, m] of the fp16 form).

    The bound, first order with a margin for what it leaves out (every term is below 2^-6 here):
      scores   an element of K rounded to fp16 (half a step each), fp32 sums of n products: dz = (2^-11 + n 2^-23) times
               sum |q k| scale; a weight is off by 2 dz relative (numerator and sum);
      weights  rounded to fp16 before their product with V, once more where the sum of the unrounded ones divides:
               2^-11 relative, 2^-25 absolute below fp16's normal range (times the positions, against a sum of >= 2^-8:
               the running maximum may lag behind by a factor of 2^8);
      values   rounded to fp16, half a step (2^-25 absolute where subnormal); fp32 sums, n 2^-23;
      output   half a step, 2^-25 where subnormal."""
    out, tol = np.zeros((len(q), V.shape[-1])), np.zeros((len(q), V.shape[-1]))
    for i in range(len(q)):
        n = first + i + 1
        if n <= 0:
            continue
        z = q[i] @ K[:n].T * scale
        dz = (np.abs(q[i]) @ np.abs(K[:n]).T * abs(scale)).max() * (HALF_STEP + K.shape[1] * 2.0 ** -23)
        p = softmax64(z)
        out[i] = p @ V[:n]
        size = p @ np.abs(V[:n])
        tol[i] = 1.05 * size * (2 * dz + 2 * HALF_STEP + (n + 64) * 2.0 ** -23 + 2.0 ** -20) + HALF_STEP * np.abs(out[i]) \
            + n * 2.0 ** -25 * 2.0 ** 8 * 2.0 ** -8 * np.abs(V[:n]).max() * p.max() + 2.0 ** -24
    return out, tol
