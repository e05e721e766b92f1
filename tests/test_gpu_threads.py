"""Calls of several host threads at once, each with its own stream, tensors and
workspace, whose launches ask for different amounts of shared memory."""
import threading

import numpy as np
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import test_gpu_evict
import test_gpu_int4_attention

pytestmark = pytest.mark.gpu

CALLS = 4000


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa.build()


def _at_once(calls):
    """Every function CALLS times on a thread of its own; what they raised."""
    raised, start = [], threading.Barrier(len(calls))

    def work(fn):
        try:
            s = torch.cuda.Stream()
            start.wait()
            for _ in range(CALLS):
                fn(s)
            s.synchronize()
        except Exception as e:                                # reported by the main thread
            raised.append(e)

    threads = [threading.Thread(target=work, args=(fn,)) for fn in calls]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return raised


def test_evictions_under_small_and_wide_tables():
    cases, calls = [], []
    for width, seed in ((40000, 60), (190000, 61), (40000, 64), (190000, 65)):
        c = test_gpu_evict.Case([300, 90], 2, 64, 16, "f16", 64, 2, 10, seed=seed, out_of_place=True)
        t = np.full((2, width // 16), -1, np.int32)
        t[:, :c.tables.shape[1]] = c.tables
        c.tables = t
        want = c.want()
        c.on_gpu()
        ws = torch.empty(pa.pa_evict_workspace_size(2, 2, t.shape[1] * 16, 64), dtype=torch.uint8, device="cuda")

        def call(s, c=c, ws=ws):
            pa.pa_evict(c.k, c.v, c.wd, c.bt, c.sl, c.nl, c.budget, num_sink=c.sink, num_recent=c.recent,
                        new_block_tables=c.nt, kept=c.kept, workspace=ws, stream=s)

        cases.append((c, want))
        calls.append(call)
    assert not _at_once(calls)
    for c, want in cases:
        c.check(want)


def test_4bit_attention_with_few_and_many_query_tokens():
    cases, calls = [], []
    for counts, seed in (([3, 2], 62), ([8, 5], 63), ([4, 4], 66), ([7, 5], 67)):    # one kernel, 24 to 64 rows per KV head
        c = test_gpu_int4_attention.Case([70, 40], 8, 1, 128, 16, "f16", seed, counts=counts).on_gpu()
        ref, out = c.run(), torch.empty_like(c.qd)
        n = pa.pa_attention_workspace_size(2, max(counts), 8, c.bt.shape[1] * 16, 128, 0)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")

        def call(s, c=c, ws=ws, out=out, m=max(counts)):
            pa.pa_attention(out, c.qd, c.k, c.v, c.bt, c.sl, c.qs, c.scale, m, "int4", workspace=ws, stream=s)

        cases.append((ref, out))
        calls.append(call)
    assert not _at_once(calls)
    for ref, out in cases:
        assert torch.equal(ref, out)


@pytest.mark.parametrize("heads", [(1, 8, 1, 8), (2, 3, 4, 5)])
def test_decode_of_different_head_counts(heads):
    """The same kernel with rings of different sizes."""
    cases, calls = [], []
    for Hkv in heads:
        g = torch.Generator().manual_seed(Hkv)
        k, v = (torch.randn(12, 16, Hkv, 128, generator=g).half().cuda() for _ in range(2))
        q = torch.randn(2, 4 * Hkv, 128, generator=g).half().cuda()
        bt = torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6)
        sl = torch.tensor([96, 41], dtype=torch.int32, device="cuda")
        ws = pa.alloc_workspace(2, 4 * Hkv, 96, 128)
        ref, out = torch.empty_like(q), torch.empty_like(q)
        pa.pa_decode(ref, q, k, v, bt, sl, 0.09, workspace=ws)

        def call(s, a=(q, k, v, bt, sl, 0.09), ws=ws, out=out):
            pa.pa_decode(out, *a, workspace=ws, stream=s)

        cases.append((ref, out))
        calls.append(call)
    assert not _at_once(calls)
    for ref, out in cases:
        assert torch.equal(ref, out)
