"""The bounded waits of attention over ragged batches of rows, made to run out on the GPU without any fault.

kvq_test_chunk_wait_timeout and kvq_test_latent_wait_timeout run the kernels with a short bound on every wait, and one
barrier of every CTA waits for an arrival that nobody makes.  The call must return soon (every copy and product it
has issued is waited for, and no phase that was never announced), raise KVQ_FLAG_WAIT_TIMEOUT, write nothing behind
the last sequence, and leave the context usable: a normal call right after it gives what the one before it gave.
"""
from __future__ import annotations

import ctypes as C

import pytest
import torch

from conftest import cuda_available
from test_rows_attention import Chunk, Latent

gpu = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]


def marked(*values):
    return [pytest.param(v, marks=gpu) for v in values]


CASES = {
    "few 128": lambda kvq: Chunk(kvq, 2, 4, 128, 16, 64, 128, [1, 3], [20000, 9000], pad=3),
    "few 64": lambda kvq: Chunk(kvq, 1, 8, 64, 32, 32, 64, [4, 0, 2], [7000, 0, 300], pad=3),
    "two row tiles": lambda kvq: Chunk(kvq, 2, 4, 128, 64, 64, 128, [200, 64], [3000, 6000], pad=3),
    "one row tile": lambda kvq: Chunk(kvq, 3, 2, 64, 16, 32, 32, [40, 33], [9000, 1], pad=3),
    "short": lambda kvq: Chunk(kvq, 1, 1, 128, 16, 64, 64, [1], [1], pad=3),
    "latent 512": lambda kvq: Latent(kvq, 512, 16, 64, 64, [1, 3], [20000, 700], pad=3),
    "latent 256": lambda kvq: Latent(kvq, 256, 100, 16, 32, [2, 9], [3000, 9], pad=3),
}


@pytest.mark.parametrize("case", marked(*CASES))
@pytest.mark.parametrize("limit", [5_000_000, 20_000, 1000])
def test_waits_run_out_and_are_flagged(kvq, case, limit):
    c = CASES[case](kvq)
    want = c.run().clone()
    assert kvq.kvq_read_status(c.ws) == 0
    fn = kvq.kvq_test_chunk_wait_timeout if isinstance(c, Chunk) else kvq.kvq_test_latent_wait_timeout
    pool, q, table, lens, cu = c.args
    before, c.out[:] = pool.clone(), 7
    t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    t0.record()
    fn(c.cfg, pool, q, table, lens, cu, c.max_len, c.scale, c.out, c.ws, limit)
    t1.record()
    t1.synchronize()
    assert kvq.kvq_read_status(c.ws) == kvq.KVQ_FLAG_WAIT_TIMEOUT
    # far below the 250 ms that a wait for a phase which never comes takes
    assert t0.elapsed_time(t1) < 100 + limit * 1e-6, t0.elapsed_time(t1)
    assert (c.out[c.cu[-1]:] == 7).all() and torch.equal(pool, before)
    c.ws[:256].zero_()
    assert torch.equal(c.run(), want) and kvq.kvq_read_status(c.ws) == 0


@pytest.mark.parametrize("latent", [False, True])
def test_limits_outside_the_range_are_refused(latent):
    from int4_group_quantized_kvq_gb300 import _build
    _build.build()
    import int4_group_quantized_kvq_gb300 as kvq
    cfg = kvq.latent_config(512, 64, 64, 64, 10) if latent else kvq.config(8, 128, 16, 64, 128, 10)
    fn = kvq.lib().kvq_test_latent_wait_timeout if latent else kvq.lib().kvq_test_chunk_wait_timeout
    args = [C.byref(cfg), 0x1000, 0x2000, 0x3000, 4, 0x4000, 0x5000, 1, 4, 16, 64, 0.1, 0x6000, 0x7000, 1 << 40]
    for limit in (0, 999, 10_000_001, 1 << 40):
        assert fn(*args, limit, None) == kvq.KVQ_EINVAL
        assert "wait_limit_ns" in kvq.kvq_last_error()
    args[1] = None
    assert fn(*args, 1000, None) == kvq.KVQ_EINVAL and "pointer" in kvq.kvq_last_error()
