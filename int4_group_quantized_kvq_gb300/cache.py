"""One layer's INT4 paged KV cache on the GPU and its decode step.

A thin holder of device buffers (torch allocates them; the library allocates
nothing) around the C ABI calls of a decode step:

    quantize-on-append of the new token's K/V  ->  kvq_quantize_append
    decode attention over the packed cache      ->  kvq_decode_attention
    both in one call (append fused in)          ->  kvq_decode_step

With ``window > 0`` the attention is restricted to the last ``window`` positions and
the first ``sinks`` (``kvq_decode_attention_window`` / ``kvq_decode_step_window``).

With ``track_weights`` the cache also accumulates the attention weight each cached position
receives (``kvq_decode_attention_weights`` / ``kvq_decode_step_weights``), and ``evict`` cuts it
by that measure to a budget of positions, each KV head keeping its own
(``kvq_evict_select``, ``kvq_evict_compact``).  A batch slot that takes a new sequence starts with
``cache.weights[b] = 0``.  ``attend_diff`` and ``decode_step_diff`` read the same pool as
differential attention, for a cache made with ``diff`` (``kvq_diff_decode_attention`` /
``kvq_diff_decode_step``); they know no window and add nothing to the weights.

Prompts, parts of prompts and drafted tokens (any number of new rows per sequence, ``cu_rows``), in a cache made
with ``rows``:
``append_rotary`` turns queries and keys by their positions and quantizes the rows into the pages
(``kvq_rope_append``), ``attend_rows`` attends with them (``kvq_chunk_attention``), ``prompt_step`` does both,
and ``read_rows`` dequantizes rows (``kvq_dequantize_varlen``).
In a cache made with ``rope`` these two, ``append_rotary`` and ``prompt_step``, are the calls that turn anything.  Every
other one (``append``, ``decode_step`` and its kin, ``HostPipeline``) stores k and uses q as they are given, so there
both must have been turned by their positions already; a decode step over projections not turned yet is
``append_rotary`` with one row per sequence (q in place), then ``attend``.

``LatentKVCache`` holds one layer's latent cache: ``step`` appends new rows (``kvq_latent_append``) and
attends in the absorbed form (``kvq_latent_attention``), for single tokens and prompts alike.

``decode_step_host`` is the same step driven from pinned host buffers (``HostStaging``)
in one kvq_decode_step_host call: the step's q, K and V are copied in with one transfer
and the output copied back, on the same stream; ``HostPipeline`` overlaps those copies
with the neighbouring steps (kvq_decode_step_host_pipelined).
"""
from __future__ import annotations

import math

import torch

from . import binding as B


class PagedKVCache:
    def __init__(self, cfg: B.CacheConfig, block_table: torch.Tensor, num_q_heads: int, max_len: int,
                 device="cuda", pool: torch.Tensor | None = None, window: int = 0, sinks: int = 0,
                 track_weights: bool = False, decay: float = 1.0, diff: bool = False,
                 rows: bool = False, rope: B.RopeConfig | None = None, cos_sin: torch.Tensor | None = None):
        self.cfg = cfg
        if (rope is None) != (cos_sin is None):
            raise ValueError("rotary positions need both rope and its table cos_sin")
        self.rope = rope
        self.cos_sin = cos_sin
        self.window = int(window)
        self.sinks = int(sinks)
        self.device = torch.device(device)
        self.block_table = block_table.to(self.device, torch.int32).contiguous()
        self.batch = int(self.block_table.shape[0])
        self.num_q_heads = int(num_q_heads)
        self.max_len = int(max_len)
        nbytes = B.kvq_pool_bytes(cfg)
        if pool is None:
            pool = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        if pool.numel() < nbytes:
            raise ValueError(f"pool has {pool.numel()} bytes, needs {nbytes}")
        self.pool = pool
        self.decay = float(decay)
        self.weights = None
        if diff and self.window > 0:
            raise ValueError("differential attention attends to every position (no window)")
        self.diff_workspace = B.new_diff_workspace(cfg, self.batch, self.num_q_heads, self.max_len,
                                                   device=self.device) if diff else None
        if rows and (self.window > 0 or track_weights):
            raise ValueError("attention of many rows attends to every position (no window) and tracks no weights")
        self.rows_workspace = B.new_chunk_workspace(cfg, self.batch, self.num_q_heads, self.max_len,
                                                    device=self.device) if rows else None
        if track_weights:
            if self.window > 0:
                raise ValueError("a cache with a window does not track weights")
            self.weights = torch.zeros(self.batch, cfg.num_kv_heads, self.max_len, dtype=torch.float32,
                                       device=self.device)
            self.workspace = B.new_weights_workspace(cfg, self.batch, self.num_q_heads, self.max_len,
                                                     device=self.device)
        else:
            self.workspace = B.new_workspace(cfg, self.batch, self.num_q_heads, self.max_len, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.softmax_scale = 1.0 / math.sqrt(cfg.head_dim)

    def append(self, k: torch.Tensor, v: torch.Tensor, start_pos: torch.Tensor, stream=None) -> None:
        """Quantize k, v [B, n, Hkv, d] fp16 into positions start_pos[b] .. start_pos[b] + n - 1 (k as it is given: where
        keys have rotary positions, turned already)."""
        B.kvq_quantize_append(self.cfg, self.pool, k, v, self.block_table, start_pos, status=self.status,
                              stream=stream)

    def attend(self, q: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor, stream=None) -> None:
        """Decode attention of q [B, Hq, d] fp16 over positions 0 .. seq_lens[b]-1 into out (fp32)."""
        if self.weights is not None:
            B.kvq_decode_attention_weights(self.cfg, self.pool, q, self.block_table, seq_lens, self.max_len,
                                           self.softmax_scale, self.decay, self.weights, out, self.workspace,
                                           stream=stream)
        elif self.window > 0:
            B.kvq_decode_attention_window(self.cfg, self.pool, q, self.block_table, seq_lens, self.max_len,
                                          self.softmax_scale, self.window, self.sinks, out, self.workspace,
                                          stream=stream)
        else:
            B.kvq_decode_attention(self.cfg, self.pool, q, self.block_table, seq_lens, self.max_len,
                                   self.softmax_scale, out, self.workspace, stream=stream)

    def decode_step(self, q, k_new, v_new, append_pos, seq_lens, out, stream=None) -> None:
        """Append one token per sequence at append_pos, then attend over seq_lens (which include it):
        one kvq_decode_step call.  q and k_new are taken as they are given: where they have rotary positions, turned
        already (for those that are not: append_rotary, then attend)."""
        if self.weights is not None:
            B.kvq_decode_step_weights(self.cfg, self.pool, k_new, v_new, append_pos, q, self.block_table, seq_lens,
                                      self.max_len, self.softmax_scale, self.decay, self.weights, out, self.workspace,
                                      stream=stream)
        elif self.window > 0:
            B.kvq_decode_step_window(self.cfg, self.pool, k_new, v_new, append_pos, q, self.block_table, seq_lens,
                                     self.max_len, self.softmax_scale, self.window, self.sinks, out, self.workspace,
                                     stream=stream)
        else:
            B.kvq_decode_step(self.cfg, self.pool, k_new, v_new, append_pos, q, self.block_table, seq_lens,
                              self.max_len, self.softmax_scale, out, self.workspace, stream=stream)

    def decode_step_two_calls(self, q, k_new, v_new, append_pos, seq_lens, out, stream=None) -> None:
        """The same step as two calls: kvq_quantize_append, then kvq_decode_attention."""
        self.append(k_new, v_new, append_pos, stream)
        self.attend(q, seq_lens, out, stream)

    def evict(self, seq_lens, keep: int, sinks: int = 0, recent: int = 0, dst_table: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
        """Cut every sequence to at most `keep` positions: the first `sinks`, the last `recent` and the ones of
        largest accumulated weight, each KV head its own.  The rows move to the front of the sequence's pages, or
        into dst_table's (int32 [B, blocks]), which then becomes the cache's block table.  dst_table has to hold the
        positions kept; a table with room for those alone is full, so a decode_step behind them appends nothing and
        flags KVQ_FLAG_BAD_POSITION on the device.  A graph captured before holds the old table's address: it is to
        be captured again, not replayed (one of this call needs the old table kept).  Returns the new lengths
        (int32 [B]); pages from ceil(new length / page_size) on are free.  Allocates its small results on the
        current stream, so `stream` is that one or one that waits for it."""
        if self.weights is None:
            raise ValueError("evict needs a cache with track_weights")
        dst = self.block_table if dst_table is None else dst_table
        pages = int(self.block_table.shape[1])  # (a sequence is no longer than its pages)
        if int(dst.shape[1]) * self.cfg.page_size < min(int(keep), self.max_len, pages * self.cfg.page_size):
            raise ValueError(f"dst_table has {int(dst.shape[1])} pages a sequence, too few for {keep} positions")
        kept = torch.empty(self.batch, self.cfg.num_kv_heads, int(keep), dtype=torch.int32, device=self.device)
        new_lens = torch.empty(self.batch, dtype=torch.int32, device=self.device)
        B.kvq_evict_select(self.cfg, self.weights, seq_lens, self.max_len, keep, sinks, recent, kept, new_lens,
                           status=self.status, stream=stream)
        B.kvq_evict_compact(self.cfg, self.pool, self.block_table, dst, seq_lens, kept, self.weights,
                            status=self.status, stream=stream)
        # no tensor's memory is handed out again before the stream has passed the calls
        if stream is not None:
            used = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
            kept.record_stream(used)
            new_lens.record_stream(used)
        if dst is not self.block_table:
            self.block_table.record_stream(torch.cuda.current_stream() if stream is None else used)
            self.block_table = dst
        return new_lens

    def attend_diff(self, q, lam, seq_lens, out, norm_weight=None, norm_eps: float = 1e-5, out_scale: float = 1.0,
                    stream=None) -> None:
        """Differential decode attention: softmax over the first halves of q and K minus lam (fp32 [Hq]) times
        softmax over the second halves, scaled by 1 / sqrt(head_dim / 2), then the optional RMS norm and scale.
        For a cache made with `diff`."""
        if self.diff_workspace is None:
            raise ValueError("attend_diff needs a cache made with diff")
        B.kvq_diff_decode_attention(self.cfg, self.pool, q, self.block_table, seq_lens, self.max_len,
                                    self.softmax_scale * math.sqrt(2.0), lam, norm_weight, norm_eps, out_scale, out,
                                    self.diff_workspace, stream=stream)

    def decode_step_diff(self, q, k_new, v_new, lam, append_pos, seq_lens, out, norm_weight=None,
                         norm_eps: float = 1e-5, out_scale: float = 1.0, stream=None) -> None:
        """Append one token per sequence at append_pos, then attend_diff over seq_lens: one kvq_diff_decode_step.  q and
        k_new are taken as they are given, as in decode_step."""
        if self.diff_workspace is None:
            raise ValueError("decode_step_diff needs a cache made with diff")
        B.kvq_diff_decode_step(self.cfg, self.pool, k_new, v_new, append_pos, q, self.block_table, seq_lens,
                               self.max_len, self.softmax_scale * math.sqrt(2.0), lam, norm_weight, norm_eps,
                               out_scale, out, self.diff_workspace, stream=stream)

    def append_rotary(self, q, k, v, q_out, start_pos, cu_rows, positions=None, stream=None) -> None:
        """Turn q into q_out (both fp16 [T, Hq, d]; the same tensor: in place) and k, and quantize k, v (fp16
        [T, Hkv, d]) into positions start_pos[b] .. of every sequence: rows cu_rows[b] .. cu_rows[b + 1] - 1 are its
        new ones.  positions (int32 [axes, T]): where the angles are taken, if not at the rows' places in the cache.
        For a cache made with rope and cos_sin.  One row per sequence, then attend: a decode step."""
        if self.rope is None:
            raise ValueError("append_rotary needs a cache made with rope and cos_sin")
        B.kvq_rope_append(self.cfg, self.rope, self.pool, q, k, v, q_out, self.cos_sin, self.block_table, start_pos, cu_rows,
                          positions=positions, status=self.status, stream=stream)

    def attend_rows(self, q, seq_lens, cu_rows, out, stream=None) -> None:
        """Causal attention of the last rows of every sequence: q fp16 [T, Hq, d] at the last positions of seq_lens
        (which include them) into out (fp16 [T, Hq, d]).  For a cache made with `rows`."""
        if self.rows_workspace is None:
            raise ValueError("attend_rows needs a cache made with rows")
        B.kvq_chunk_attention(self.cfg, self.pool, q, self.block_table, seq_lens, cu_rows, self.max_len, self.softmax_scale,
                              out, self.rows_workspace, stream=stream)

    def prompt_step(self, q, k, v, start_pos, seq_lens, cu_rows, out, positions=None, stream=None) -> None:
        """New rows of every sequence, a prompt or a part of one: append_rotary (q in place), then attend_rows;
        without rope, kvq_quantize_append_varlen in its place.  seq_lens[b] = start_pos[b] + new rows."""
        if self.rope is not None:
            self.append_rotary(q, k, v, q, start_pos, cu_rows, positions, stream)
        else:
            B.kvq_quantize_append_varlen(self.cfg, self.pool, k, v, self.block_table, start_pos, cu_rows, status=self.status,
                                         stream=stream)
        self.attend_rows(q, seq_lens, cu_rows, out, stream)

    def read_rows(self, start_pos, cu_rows, out_k, out_v, stream=None) -> None:
        """Positions start_pos[b] .. of every sequence, dequantized into out_k, out_v (fp16 or fp32 [T, Hkv, d])."""
        B.kvq_dequantize_varlen(self.cfg, self.pool, self.block_table, start_pos, cu_rows, out_k, out_v,
                                status=self.status, stream=stream)

    def decode_step_host(self, staging: "HostStaging", append_pos, seq_lens, stream=None) -> None:
        """The decode step from pinned host memory in one kvq_decode_step_host call: one H2D copy of
        the step's q, K and V (staged back to back, taken as they are given: decode_step), the step, one
        D2H copy of the output, all asynchronous on the step's stream."""
        if self.window > 0:
            raise ValueError("the host step attends to every position (no window)")
        if self.weights is not None:
            raise ValueError("the host step does not track weights")
        B.kvq_decode_step_host(self.cfg, self.pool, staging.host, staging.dev, append_pos, self.block_table, seq_lens,
                               self.batch, self.num_q_heads, self.max_len, self.softmax_scale, staging.out,
                               staging.out_host, self.workspace, stream=stream)

    def flags(self) -> int:
        """Status flags of the last calls (synchronizes)."""
        f = B.kvq_read_status(self.status) | B.kvq_read_status(self.workspace)
        if self.rows_workspace is not None:
            f |= B.kvq_read_status(self.rows_workspace)
        return f if self.diff_workspace is None else f | B.kvq_read_status(self.diff_workspace)


class LatentKVCache:
    """One layer's latent cache: pages of 4-bit latents and fp16 rotary keys, one row per token for all heads."""

    def __init__(self, cfg: B.LatentConfig, block_table: torch.Tensor, num_heads: int, max_len: int, rope: B.RopeConfig,
                 cos_sin: torch.Tensor, softmax_scale: float, norm_weight: torch.Tensor | None = None,
                 norm_eps: float = 1e-6, device="cuda", pool: torch.Tensor | None = None):
        self.cfg = cfg
        self.device = torch.device(device)
        self.block_table = block_table.to(self.device, torch.int32).contiguous()
        self.batch = int(self.block_table.shape[0])
        self.num_heads = int(num_heads)
        self.max_len = int(max_len)
        self.rope, self.cos_sin = rope, cos_sin
        self.softmax_scale = float(softmax_scale)
        self.norm_weight, self.norm_eps = norm_weight, float(norm_eps)
        nbytes = B.kvq_latent_pool_bytes(cfg)
        self.pool = torch.zeros(nbytes, dtype=torch.uint8, device=self.device) if pool is None else pool
        if self.pool.numel() < nbytes:
            raise ValueError(f"pool has {self.pool.numel()} bytes, needs {nbytes}")
        self.workspace = B.new_latent_workspace(cfg, self.batch, self.num_heads, self.max_len, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

    def append(self, rows, q_pe, q, start_pos, cu_rows, positions=None, stream=None) -> None:
        """New rows (fp16 [T, L + R]: latent, rotary key) of every sequence into positions start_pos[b] ..; q_pe (fp16
        [T, H, R]) turned into the last R values of q (fp16 [T, H, L + R]), or both None."""
        B.kvq_latent_append(self.cfg, self.rope, self.pool, rows, self.norm_weight, self.norm_eps, q_pe, q, self.cos_sin,
                            self.block_table, start_pos, cu_rows, positions=positions, status=self.status, stream=stream)

    def attend(self, q, seq_lens, cu_rows, out, stream=None) -> None:
        """Attention in the absorbed form: q fp16 [T, H, L + R] at the last positions of seq_lens, out fp16 [T, H, L]."""
        B.kvq_latent_attention(self.cfg, self.pool, q, self.block_table, seq_lens, cu_rows, self.max_len,
                               self.softmax_scale, out, self.workspace, stream=stream)

    def step(self, rows, q_pe, q, start_pos, seq_lens, cu_rows, out, positions=None, stream=None) -> None:
        """append, then attend: a decode step with one row per sequence, a prompt with many."""
        self.append(rows, q_pe, q, start_pos, cu_rows, positions, stream)
        self.attend(q, seq_lens, cu_rows, out, stream)

    def read_rows(self, start_pos, cu_rows, out, stream=None) -> None:
        """Rows read back into out (fp16 [T, L + R]), for the expanded form's matrix products."""
        B.kvq_latent_dequantize(self.cfg, self.pool, self.block_table, start_pos, cu_rows, out, status=self.status,
                                stream=stream)

    def flags(self) -> int:
        """Status flags of the last calls (synchronizes)."""
        return B.kvq_read_status(self.status) | B.kvq_read_status(self.workspace)


class HostStaging:
    """Pinned host buffers and their device twins for one decode step: q [B, Hq, d], k_new and
    v_new [B, Hkv, d] fp16 back to back (so a step copies its inputs in one transfer), and the
    fp32 output [B, Hq, d].  Fill `q_host`, `k_host`, `v_host` on the host; read `out_host`
    after the stream has passed the step."""

    def __init__(self, batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, device="cuda"):
        nq = batch * num_q_heads * head_dim
        nk = batch * num_kv_heads * head_dim
        self.host = torch.empty(nq + 2 * nk, dtype=torch.float16).pin_memory()
        self.dev = torch.empty(nq + 2 * nk, dtype=torch.float16, device=device)
        shq = (batch, num_q_heads, head_dim)
        shk = (batch, num_kv_heads, head_dim)
        self.q_host = self.host[:nq].view(shq)
        self.k_host = self.host[nq:nq + nk].view(shk)
        self.v_host = self.host[nq + nk:].view(shk)
        self.q = self.dev[:nq].view(shq)
        self.k_new = self.dev[nq:nq + nk].view(shk)
        self.v_new = self.dev[nq + nk:].view(shk)
        self.out = torch.empty(shq, dtype=torch.float32, device=device)
        self.out_host = torch.empty(shq, dtype=torch.float32).pin_memory()


class HostPipeline:
    """Decode steps fed from pinned host memory with the copies overlapped with the kernels:
    one kvq_decode_step_host_pipelined call per step.

    Two staging slots alternate.  Step i (slot i % 2) copies its inputs host-to-device on an
    input copy stream, runs on the compute stream once that copy is done, and copies its
    output device-to-host on an output copy stream once the step is done; so step i + 1's
    inputs move while step i computes, and step i's output moves while step i + 1 computes.
    The slot's three events (input copied, step done, output copied) keep its device buffers
    from being overwritten while in use: a slot's input copy waits for the step two back to
    have read that slot, and its step waits for that step's output copy to have left the slot.
    The host side is the caller's: fill `slot(i)`'s host inputs before `step(i)` (for i >= 2,
    after `inputs_copied(i - 2)`), and read its `out_host` after `done(i)` and before
    `step(i + 2)`."""

    def __init__(self, cache: PagedKVCache, compute_stream=None):
        self.cache = cache
        dev = cache.device
        self.slots = [HostStaging(cache.batch, cache.num_q_heads, cache.cfg.num_kv_heads, cache.cfg.head_dim, dev)
                      for _ in range(2)]
        self.compute = torch.cuda.Stream(device=dev) if compute_stream is None else compute_stream
        self.copy_in = torch.cuda.Stream(device=dev)
        self.copy_out = torch.cuda.Stream(device=dev)
        # per slot: input copied, step done, output copied; recorded once so that they exist
        self.events = [[torch.cuda.Event() for _ in range(3)] for _ in range(2)]
        for evs in self.events:
            for ev in evs:
                ev.record(self.compute)
        self.compute.synchronize()

    def slot(self, i: int) -> HostStaging:
        return self.slots[i % 2]

    def step(self, i: int, append_pos: torch.Tensor, seq_lens: torch.Tensor, cache: PagedKVCache | None = None) -> None:
        """Step i on `cache` (default: the pipeline's), from slot(i)'s host inputs to its out_host."""
        cache = self.cache if cache is None else cache
        st = self.slots[i % 2]
        if cache.window > 0:
            raise ValueError("the pipelined host step attends to every position (no window)")
        if cache.weights is not None:
            raise ValueError("the pipelined host step does not track weights")
        B.kvq_decode_step_host_pipelined(cache.cfg, cache.pool, st.host, st.dev, append_pos, cache.block_table,
                                         seq_lens, cache.batch, cache.num_q_heads, cache.max_len,
                                         cache.softmax_scale, st.out, st.out_host, cache.workspace, self.compute,
                                         self.copy_in, self.copy_out, self.events[i % 2])

    def inputs_copied(self, i: int) -> torch.cuda.Event:
        """The event after which step i's host inputs have been read (slot(i) may be refilled)."""
        return self.events[i % 2][0]

    def done(self, i: int) -> torch.cuda.Event:
        """The event after which step i's output is in slot(i).out_host (until step i + 2 is issued)."""
        return self.events[i % 2][2]

    def synchronize(self) -> None:
        for s in (self.copy_in, self.compute, self.copy_out):
            s.synchronize()
