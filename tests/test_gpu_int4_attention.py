"""Attention over 4-bit pools (pa_decode, pa_attention, pa_decode_noalloc)
against the formulas in 64 bits on the values that the pools hold."""
import numpy as np
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _int4
from test_gpu_guards import guarded_like, guards_intact

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa.build()


class Case:
    """Pools, tables and queries of a batch; every slot no token owns reads as NaN."""

    def __init__(self, lens, Hq, Hkv, D, bs, dtype, seed, counts=None, k_mult=1.0, v_mult=1.0, max_blocks=None,
                 q_mult=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.dtype, self.D, self.bs, self.counts = list(lens), dtype, D, bs, counts
        self.tables, self.NB, used = _int4.tables_for(rng, lens, bs, max_blocks=max_blocks)
        self.pools = [_int4.poison(p, used) for p in _int4.random_pools(rng, self.NB, bs, Hkv, D, k_mult, v_mult)]
        rows = len(lens) if counts is None else sum(counts)
        self.q = torch.from_numpy(rng.standard_normal((rows, Hq, D)) * q_mult).to(DT[dtype])
        self.scale = 1 / np.sqrt(D) / max(1.0, k_mult * q_mult)
        self.q_start = None if counts is None else np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)

    def want(self):
        return _int4.attention(self.q.double().numpy(), self.pools, self.tables, self.lens, self.scale, self.q_start,
                               self.dtype)

    def on_gpu(self):
        self.k, self.v = (torch.from_numpy(p).cuda() for p in self.pools)
        self.bt, self.sl = torch.from_numpy(self.tables).cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.qd, self.err = self.q.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
        self.qs = None if self.q_start is None else torch.from_numpy(self.q_start).cuda()
        return self

    def run(self, pt=0, workspace=None, out=None, fn=None):
        out = torch.full_like(self.qd, float("nan")) if out is None else out
        kw = dict(partition_tokens=pt, err_flag=self.err)
        if self.qs is not None:
            pa.pa_attention(out, self.qd, self.k, self.v, self.bt, self.sl, self.qs, self.scale, max(self.counts),
                            "int4", workspace=workspace, **kw)
        elif fn is not None:
            fn(out, self.qd, self.k, self.v, self.bt, self.sl, self.scale, "int4", **kw)
        else:
            pa.pa_decode(out, self.qd, self.k, self.v, self.bt, self.sl, self.scale, "int4", workspace=workspace, **kw)
        torch.cuda.synchronize()
        return out


def check(got, want, tol):
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all()
    off = np.abs(g - want) - tol
    assert (off <= 0).all(), f"{(off > 0).sum()} of {off.size} beyond the bound, worst {off.max():.3g}"


DECODE = [
    # lens, Hq, Hkv, D, bs, dtype
    ([1], 1, 1, 64, 8, "f16"),
    ([5, 16, 17, 40], 4, 2, 64, 16, "f16"),
    ([0, 1, 15, 0, 64, 65, 63], 8, 8, 128, 16, "bf16"),
    ([300, 17, 900, 5, 128], 28, 4, 128, 16, "f16"),
    ([777, 64, 1, 2049], 32, 8, 128, 32, "bf16"),
    ([250, 31, 33], 7, 1, 128, 8, "bf16"),
    ([513, 12], 6, 3, 64, 64, "bf16"),
    ([1000, 129, 127], 16, 2, 128, 128, "f16"),
    ([400, 399], 12, 1, 128, 16, "f16"),
    ([97, 201], 32, 2, 64, 32, "f16"),
    ([333], 64, 1, 128, 16, "bf16"),
    ([150, 90], 128, 1, 64, 8, "f16"),
    ([5000], 8, 2, 128, 16, "bf16"),
    ([70, 71], 10, 10, 128, 16, "f16"),
]


@pytest.mark.parametrize("pt", [0, 64, 48])
@pytest.mark.parametrize("k", range(len(DECODE)))
def test_decode(k, pt):
    c = Case(*DECODE[k], seed=100 + k).on_gpu()
    check(c.run(pt), *c.want())
    assert c.err.item() == 0


def test_many_short_sequences():
    rng = np.random.default_rng(3)
    c = Case(rng.integers(0, 90, 700), 8, 2, 128, 16, "bf16", seed=4).on_gpu()
    check(c.run(), *c.want())


def test_one_long_sequence_over_every_cta():
    c = Case([40007], 8, 4, 128, 32, "f16", seed=5).on_gpu()
    check(c.run(), *c.want())
    check(c.run(512), *c.want())


def test_table_wider_than_any_sequence():
    c = Case([100, 3], 8, 2, 64, 16, "f16", seed=6, max_blocks=64).on_gpu()
    check(c.run(), *c.want())


@pytest.mark.parametrize("k_mult,v_mult,q_mult", [(1e-3, 1e-3, 1.0), (30.0, 1e-5, 1.0), (1.0, 2000.0, 1e-2),
                                                  (1.0, 1.0, 300.0)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_magnitudes(k_mult, v_mult, q_mult, dtype):
    """Steps below the smallest normal f16, and values near its largest."""
    c = Case([130, 700, 31], 8, 2, 128, 16, dtype, seed=7, k_mult=k_mult, v_mult=v_mult, q_mult=q_mult).on_gpu()
    check(c.run(), *c.want())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_value_steps_that_grow_and_shrink_along_a_sequence(dtype):
    """Rows whose steps differ by 2^20 and more, in both orders, equal rows (step 0) among them."""
    c = Case([600, 600], 8, 2, 128, 16, dtype, seed=8)
    for i in range(2):
        code, step, low = _int4.rows(c.pools[1])
        code, step, low = code.copy(), step.copy(), low.copy()
        pos = np.arange(600)
        b, o = c.tables[i][pos // 16], pos % 16
        f = (2.0 ** (np.where(i == 0, pos, 599 - pos) / 30.0 - 10))[:, None]
        step[b, o] = (step[b, o].astype(np.float64) * f).astype(np.float16)
        low[b, o] = (low[b, o].astype(np.float64) * f).astype(np.float16)
        step[b[100:140], o[100:140]] = 0
        c.pools[1] = _int4.pack(code, step, low)
    c.on_gpu()
    check(c.run(), *c.want())


def test_a_needle_decides_the_output():
    """One key that takes nearly all weight, anywhere in the sequence."""
    c = Case([500, 129, 64], 8, 2, 128, 16, "f16", seed=9)
    code, step, low = (x.copy() for x in _int4.rows(c.pools[0]))
    for i, t in enumerate((499, 0, 37)):
        b, o = c.tables[i][t // 16], t % 16
        for g in range(2):
            k = c.q[i, 4 * g].double().numpy() * 3
            code[b, o, g], step[b, o, g], low[b, o, g] = (x[0] for x in _int4.encode(k[None]))
    c.pools[0] = _int4.pack(code, step, low)
    c.on_gpu()
    check(c.run(), *c.want())


def test_a_row_that_holds_nan_reaches_only_its_own_head():
    c = Case([100, 50], 4, 2, 64, 16, "f16", seed=10)
    code, step, low = (x.copy() for x in _int4.rows(c.pools[1]))
    b, o = c.tables[0][3], 5
    step[b, o, 1] = low[b, o, 1] = np.float16("nan")
    pools = [c.pools[0], _int4.pack(code, step, low)]
    want, tol = c.want()
    c.pools = pools
    got = c.on_gpu().run()
    assert torch.isnan(got[0, 2:]).all()
    got[0, 2:] = torch.from_numpy(want[0, 2:]).to(got)
    check(got, want, tol)


MULTI = [
    # lens, counts, Hq, Hkv, D, bs, dtype
    ([20, 300, 7], [3, 1, 4], 4, 2, 64, 16, "f16"),
    ([64, 200, 40], [4, 4, 2], 28, 4, 128, 16, "f16"),
    ([1000, 30, 500], [8, 5, 1], 32, 8, 128, 32, "bf16"),
    ([100, 0, 2, 90], [2, 3, 5, 0], 8, 1, 128, 8, "bf16"),     # no keys, fewer keys than queries, no queries
    ([700, 128], [16, 16], 8, 1, 128, 16, "bf16"),              # 128 rows
    ([128, 65], [31, 7], 16, 4, 64, 128, "f16"),
    ([50, 50], [9, 9], 14, 2, 128, 16, "f16"),
]


@pytest.mark.parametrize("pt", [0, 64])
@pytest.mark.parametrize("k", range(len(MULTI)))
def test_attention(k, pt):
    lens, counts, Hq, Hkv, D, bs, dtype = MULTI[k]
    c = Case(lens, Hq, Hkv, D, bs, dtype, seed=200 + k, counts=counts).on_gpu()
    check(c.run(pt), *c.want())
    assert c.err.item() == 0


def test_attention_over_a_long_sequence():
    c = Case([20011, 17], 16, 4, 128, 16, "f16", seed=21, counts=[6, 2]).on_gpu()
    check(c.run(), *c.want())


def test_one_query_token_equals_decode():
    c = Case([300, 17, 900], 28, 4, 128, 16, "f16", seed=22, counts=[1, 1, 1]).on_gpu()
    a = c.run()
    c.qs = None
    assert torch.equal(a, c.run())


def test_repeats_and_a_used_workspace_give_the_same_bits():
    c = Case([3000, 17, 900, 64], 28, 4, 128, 16, "f16", seed=23).on_gpu()
    ref = c.run()
    ws = torch.full((pa.pa_decode_workspace_size(4, 28, c.bt.shape[1] * 16, 128, 0),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    for _ in range(3):
        assert torch.equal(c.run(workspace=ws), ref)
    d = Case([64, 64], 8, 2, 64, 16, "bf16", seed=24).on_gpu()
    check(d.run(workspace=ws), *d.want())
    assert torch.equal(c.run(workspace=ws), ref)


def test_noalloc_equals_decode():
    c = Case([3000, 9000, 17], 32, 8, 128, 32, "bf16", seed=25).on_gpu()
    assert torch.equal(c.run(fn=pa.pa_decode_noalloc), c.run())


def test_output_and_workspace_stay_in_bounds():
    for counts, pt in ((None, 0), (None, 64), ([3, 1, 5], 0)):
        c = Case([300, 17, 900], 12, 3, 128, 16, "bf16", seed=26, counts=counts).on_gpu()
        MB = c.bt.shape[1] * 16
        n = pa.pa_decode_workspace_size(3, 12, MB, 128, pt) if counts is None else \
            pa.pa_attention_workspace_size(3, 5, 12, MB, 128, pt)
        wbuf, ws = guarded_like(torch.zeros(n, dtype=torch.uint8, device="cuda"))
        obuf, out = guarded_like(torch.zeros_like(c.qd))
        c.run(pt, ws, out)
        assert guards_intact(wbuf) and guards_intact(obuf)
        assert torch.equal(out, c.run(pt))


def test_graph_replay_and_another_stream():
    c = Case([700, 20, 64], 8, 2, 128, 16, "f16", seed=27).on_gpu()
    ref = c.run()
    ws = pa.alloc_workspace(3, 8, c.bt.shape[1] * 16, 128)
    x = torch.randn(3, 2, 128, device="cuda").half()
    slots = torch.from_numpy(np.array([c.tables[i][(L - 1) // 16] * 16 + (L - 1) % 16
                                       for i, L in enumerate(c.lens)], dtype=np.int64)).cuda()

    def step(out):
        pa.pa_reshape_and_cache(c.k, c.v, x, x, slots, "int4")
        pa.pa_decode(out, c.qd, c.k, c.v, c.bt, c.sl, c.scale, "int4", workspace=ws)

    want = torch.empty_like(ref)
    step(want)
    torch.cuda.synchronize()
    assert not torch.equal(want, ref)
    out = torch.zeros_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    s = torch.cuda.Stream()
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    pa.pa_decode(out, c.qd, c.k, c.v, c.bt, c.sl, c.scale, "int4", workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_bad_blocks_and_lengths_are_flagged():
    c = Case([100, 60, 40], 8, 2, 64, 16, "f16", seed=28)
    keep = c.tables.copy()
    c.tables[1, 2] = c.NB + 3
    c.on_gpu()
    got = c.run()
    assert c.err.item() == pa.ERRBIT_BAD_BLOCK
    c.tables = keep
    want, tol = c.want()
    check(got[[0, 2]], want[[0, 2]], tol[[0, 2]])
    # the bad block's 16 tokens are left out
    t = _int4.rows(c.pools[0])[0].shape
    assert t[1] == 16
    lens = [100, 44, 40]
    c.tables[1, 2] = c.tables[1, 3]
    c.lens = lens
    want, tol = c.want()
    check(got[[1]], want[[1]], tol[[1]])
    c.tables = keep
    c.lens = [100, 60, 5000]                        # longer than its table: its table's tokens, and a flag
    c.on_gpu()
    c.run()
    assert c.err.item() & pa.ERRBIT_SEQ_TOO_LONG


def test_bad_query_offsets_skip_the_sequence():
    c = Case([100, 60, 40], 8, 2, 64, 16, "f16", seed=29, counts=[2, 6, 3]).on_gpu()
    want, tol = c.want()
    out = torch.full_like(c.qd, 5.0)
    pa.pa_attention(out, c.qd, c.k, c.v, c.bt, c.sl, c.qs, c.scale, 4, "int4", err_flag=c.err)
    torch.cuda.synchronize()
    assert c.err.item() == pa.ERRBIT_BAD_QUERY
    assert (out[2:8] == 5.0).all()
    rows = [0, 1, 8, 9, 10]
    check(out[rows], want[rows], tol[rows])


def test_two_calls_at_once_with_a_workspace_each():
    a = Case([3000, 100, 700], 28, 4, 128, 16, "f16", seed=30).on_gpu()
    b = Case([2000, 2001], 8, 2, 128, 32, "bf16", seed=31, counts=[3, 5]).on_gpu()
    ra, rb = a.run(), b.run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    wa = pa.alloc_workspace(3, 28, a.bt.shape[1] * 16, 128)
    wb = torch.empty(pa.pa_attention_workspace_size(2, 5, 8, b.bt.shape[1] * 32, 128, 0), dtype=torch.uint8, device="cuda")
    oa, ob = torch.zeros_like(ra), torch.zeros_like(rb)
    torch.cuda.synchronize()
    for _ in range(20):
        pa.pa_decode(oa, a.qd, a.k, a.v, a.bt, a.sl, a.scale, "int4", workspace=wa, stream=streams[0])
        pa.pa_attention(ob, b.qd, b.k, b.v, b.bt, b.sl, b.qs, b.scale, 5, "int4", workspace=wb, stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(oa, ra) and torch.equal(ob, rb)


def test_many_heads_and_a_group_of_nine():
    """More KV heads than CTAs per range, and groups just over the 8 rows of a warp."""
    c = Case([40, 300], 256, 256, 64, 8, "f16", seed=32).on_gpu()
    check(c.run(), *c.want())
    c = Case([200, 33], 27, 3, 128, 16, "bf16", seed=33).on_gpu()
    check(c.run(), *c.want())


def test_an_infinite_query_element_spoils_only_its_head():
    c = Case([100, 70], 4, 2, 64, 16, "f16", seed=34)
    want, tol = c.want()
    c.q[0, 1, 3] = float("inf")
    got = c.on_gpu().run()
    assert not torch.isfinite(got[0, 1]).all()
    got[0, 1] = torch.from_numpy(want[0, 1]).to(got)
    check(got, want, tol)


@pytest.mark.parametrize("wide", [1, 40])
@pytest.mark.parametrize("lens", [[1], [5000, 12000, 17001], [129, 0, 260, 1], [39000]])
def test_fewer_chunks_than_ranges(lens, wide):
    """Few long sequences of one KV head, also under tables for many more tokens."""
    c = Case(lens, 7, 1, 128, 32, "f16", seed=35)
    if wide > 1:
        t = np.full((len(lens), c.tables.shape[1] * wide), -1, np.int32)
        t[:, :c.tables.shape[1]] = c.tables
        c.tables = t
    check(c.on_gpu().run(), *c.want())
