"""pa_evict against the definition, every byte of the pools and weights, in
place and into other blocks."""
import numpy as np
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _evict
import _int4
from test_gpu_guards import guarded_like, guards_intact

pytestmark = pytest.mark.gpu

ELEM = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "fp8_e4m3": torch.uint8,
        "fp8_e5m2": torch.float8_e5m2, "int4": torch.uint8}
WIDTH = {"f32": 4, "f16": 2, "bf16": 2, "fp8_e4m3": 1, "fp8_e5m2": 1}


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa.build()


class Case:
    def __init__(self, lens, Hkv, D, bs, kv, budget, sink, recent, seed, weights="heavy", out_of_place=False):
        rng = np.random.default_rng(seed)
        self.lens, self.Hkv, self.D, self.bs, self.kv = list(lens), Hkv, D, bs, kv
        self.budget, self.sink, self.recent = budget, sink, recent
        both = list(lens) + ([min(L, budget) for L in lens] if out_of_place else [])
        tables, self.NB, _ = _int4.tables_for(rng, both, bs)
        self.tables = tables[:len(lens)]
        self.new_tables = tables[len(lens):, :max(1, -(-budget // bs))].copy() if out_of_place else None
        row = D // 2 + 4 if kv == "int4" else D * WIDTH[kv]
        self.pools = [rng.integers(0, 256, (self.NB, bs, Hkv, row)).astype(np.uint8) for _ in range(2)]
        w = np.exp(2 * rng.standard_normal((self.NB, Hkv, bs))).astype(np.float32)
        if weights == "ties":
            w = rng.integers(0, 3, w.shape).astype(np.float32)
        elif weights == "equal":
            w[:] = 0.25
        elif weights == "odd":                     # NaN, infinities, signed zeros, negatives, subnormals
            w = rng.choice(np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, -1.5, 1e-42, -1e-42, 3.0, 1.0, 1.0000001],
                                    np.float32), w.shape)
        self.w = w.astype(np.float32)

    def rows(self, pool):
        """[NB, bs, Hkv, row bytes] whatever the layout inside a block."""
        if self.kv != "int4":
            return pool
        codes, par = _int4.split(pool)
        return np.concatenate([codes, par.view(np.uint8).reshape(par.shape[:3] + (4,))], -1).transpose(0, 2, 1, 3)

    def want(self):
        return _evict.evict([self.rows(p) for p in self.pools], self.w, self.tables, self.lens, self.budget, self.sink,
                            self.recent, self.bs, None, self.new_tables)

    def on_gpu(self):
        if self.kv == "int4":
            self.k, self.v = (torch.from_numpy(p).cuda() for p in self.pools)
        else:
            self.k, self.v = (torch.from_numpy(p).cuda().view(ELEM[self.kv]).view(self.NB, self.bs, self.Hkv, self.D)
                              for p in self.pools)
        self.wd, self.bt = torch.from_numpy(self.w).cuda(), torch.from_numpy(self.tables).cuda()
        self.nt = None if self.new_tables is None else torch.from_numpy(self.new_tables).cuda()
        self.sl = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.nl = torch.full_like(self.sl, -7)
        self.kept = torch.full((len(self.lens), self.Hkv, self.budget), -9, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self

    def run(self, **kw):
        pa.pa_evict(self.k, self.v, self.wd, self.bt, self.sl, self.nl, self.budget, self.kv, num_sink=self.sink,
                    num_recent=self.recent, new_block_tables=self.nt, **{"kept": self.kept, "err_flag": self.err, **kw})
        torch.cuda.synchronize()
        return self

    def check(self, want=None):
        pools, w, lens, kept = want or self.want()
        assert np.array_equal(self.nl.cpu().numpy(), lens)
        assert np.array_equal(self.kept.cpu().numpy(), kept)
        assert np.array_equal(self.wd.cpu().numpy().view(np.uint32), w.view(np.uint32))
        for got, p in zip((self.k, self.v), pools):
            got = got.contiguous().view(torch.uint8).cpu().numpy().reshape(self.pools[0].shape)
            assert np.array_equal(self.rows(got), p)


SHAPES = [
    # lens, Hkv, D, bs, kv, budget, sink, recent
    ([33], 1, 64, 8, "f16", 32, 0, 0),
    ([100, 17, 64, 65, 0, 1], 2, 64, 16, "f16", 64, 4, 16),
    ([300, 40, 90], 3, 128, 16, "bf16", 48, 0, 48),               # the recent ones alone
    ([300, 129], 2, 128, 32, "f32", 128, 0, 0),                    # the heavy ones alone
    ([130, 128, 127], 8, 128, 32, "int4", 100, 3, 31),
    ([500, 90], 4, 64, 64, "int4", 64, 1, 7),
    ([257, 250], 2, 128, 128, "fp8_e4m3", 250, 8, 240),            # no room for a heavy one
    ([77, 200, 90], 5, 64, 8, "fp8_e5m2", 40, 40, 0),              # sinks alone
    ([400, 399], 1, 128, 16, "f16", 398, 0, 300),                  # few rows go, a long shift by one and by two
    ([50, 3], 2, 64, 16, "f16", 1, 0, 0),
    ([50, 3], 2, 64, 16, "f16", 1, 0, 1),
    ([2064, 2064], 4, 128, 16, "f16", 2048, 4, 256),
    ([5000, 700], 2, 128, 16, "bf16", 600, 4, 64),
    ([900, 1024, 1025], 2, 64, 32, "f16", 1023, 5, 500),
]


@pytest.mark.parametrize("out_of_place", [False, True])
@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_evict(k, out_of_place):
    c = Case(*SHAPES[k], seed=300 + k, out_of_place=out_of_place)
    c.on_gpu().run().check()
    assert c.err.item() == 0


@pytest.mark.parametrize("weights", ["ties", "equal", "odd"])
@pytest.mark.parametrize("out_of_place", [False, True])
def test_weights_that_tie_or_are_no_numbers(weights, out_of_place):
    c = Case([700, 65, 200], 3, 64, 16, "f16", 64, 2, 10, seed=31, weights=weights, out_of_place=out_of_place)
    c.on_gpu().run().check()


def test_a_long_sequence():
    c = Case([70001, 40], 1, 64, 32, "f16", 4100, 4, 512, seed=32, weights="ties")
    c.on_gpu().run().check()


@pytest.mark.parametrize("weights", ["heavy", "ties"])
@pytest.mark.parametrize("width", [20000, 60000, 150000, 210000])
def test_tables_for_more_tokens_than_any_sequence_has(weights, width):
    """The selection is cut over 1 to 8 CTAs, and its keys kept or read again, by what the tables could hold."""
    c = Case([3000, 40, 1201], 2, 64, 16, "f16", 500, 4, 100, seed=41, weights=weights)
    wide = np.full((3, width // 16), -1, np.int32)
    wide[:, :c.tables.shape[1]] = c.tables
    c.tables = wide
    c.on_gpu().run().check()
    assert c.err.item() == 0


@pytest.mark.parametrize("weights", ["heavy", "ties", "equal"])
@pytest.mark.parametrize("budget,out_of_place", [(5000, False), (150007, False), (5000, True)])
def test_long_runs_of_one_thread(weights, budget, out_of_place):
    """47 keys of one thread, the sinks and the place where the recent rows go inside such a run."""
    c = Case([190001], 1, 16, 32, "f16", budget, 40, 1003, seed=46, weights=weights, out_of_place=out_of_place)
    c.on_gpu().run().check()


def test_one_row_over_a_whole_cluster():
    c = Case([30000], 1, 64, 32, "f16", 29000, 7, 3000, seed=42, weights="ties")
    c.on_gpu().run().check()


def test_many_sequences():
    rng = np.random.default_rng(33)
    c = Case(rng.integers(0, 150, 300), 2, 64, 16, "f16", 64, 1, 9, seed=34)
    c.on_gpu().run().check()


def test_lengths_written_over_and_no_kept_positions():
    c = Case([100, 17, 300], 2, 64, 16, "bf16", 64, 4, 16, seed=35).on_gpu()
    want = c.want()
    c.nl = c.sl
    c.run(kept=None)
    c.kept = torch.from_numpy(want[3])
    c.check(want)


def test_twice_in_place_keeps_the_recent_rows_last():
    """A second eviction after ten more tokens: positions of the first call's result."""
    c = Case([200, 150], 2, 64, 16, "f16", 64, 2, 20, seed=36).on_gpu()
    c.run()
    c.check()
    lens = [74, 74]
    c.lens = lens
    c.pools = [x.contiguous().view(torch.uint8).cpu().numpy().reshape(c.pools[0].shape) for x in (c.k, c.v)]
    c.w = c.wd.cpu().numpy()
    c.on_gpu().run().check()


def test_guards_and_a_garbage_workspace():
    for oop in (False, True):
        c = Case([300, 20, 129], 3, 64, 16, "int4", 64, 2, 10, seed=37, out_of_place=oop).on_gpu()
        ws = torch.full((pa.pa_evict_workspace_size(3, 3, c.bt.shape[1] * 16, 64),), 0xEE, dtype=torch.uint8, device="cuda")
        bufs = []
        for name in ("k", "v", "wd", "kept", "nl"):
            b, x = guarded_like(getattr(c, name))
            bufs.append(b)
            setattr(c, name, x)
        wb, ws = guarded_like(ws)
        c.run(workspace=ws)
        c.check()
        assert all(guards_intact(b) for b in bufs + [wb])


def test_graph_replay_and_another_stream():
    c = Case([300, 70], 2, 64, 16, "f16", 64, 2, 10, seed=38, out_of_place=True).on_gpu()
    ws = torch.empty(pa.pa_evict_workspace_size(2, 2, c.bt.shape[1] * 16, 64), dtype=torch.uint8, device="cuda")
    want = c.want()
    c.run(workspace=ws).check(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_evict(c.k, c.v, c.wd, c.bt, c.sl, c.nl, c.budget, num_sink=c.sink, num_recent=c.recent,
                    new_block_tables=c.nt, kept=c.kept, workspace=ws)
    c.kept.fill_(-9)
    c.nl.fill_(-7)
    graph.replay()
    torch.cuda.synchronize()
    c.check(want)
    s = torch.cuda.Stream()
    c.kept.fill_(-9)
    s.wait_stream(torch.cuda.current_stream())
    c.run(workspace=ws, stream=s)
    s.synchronize()
    c.check(want)


def test_bad_sequences_are_skipped():
    for oop in (False, True):
        c = Case([100, 90, 200, 80], 2, 64, 16, "f16", 64, 2, 10, seed=39, out_of_place=oop)
        want = c.want()
        c.tables = c.tables.copy()
        c.tables[1, 3] = c.NB
        c.on_gpu()
        c.sl[2] = 16 * c.bt.shape[1] + 1
        c.run()
        assert c.err.item() == pa.ERRBIT_BAD_BLOCK | pa.ERRBIT_SEQ_TOO_LONG
        # sequences 1 and 2 as they were
        ref = Case([100, 0, 0, 80], 2, 64, 16, "f16", 64, 2, 10, seed=39, out_of_place=False)
        ref.tables = np.where(c.tables < c.NB, c.tables, 0)
        ref.NB, ref.pools, ref.w, ref.new_tables = c.NB, c.pools, c.w, c.new_tables
        pools, w, lens, kept = ref.want()
        lens = lens.copy()
        lens[1:3] = 0 if oop else (90, 16 * c.bt.shape[1] + 1)
        c.check((pools, w, lens, kept))
        assert np.array_equal(kept[0], want[3][0])


def test_new_tables_too_narrow_or_outside_the_pool():
    c = Case([100, 90], 2, 64, 16, "f16", 64, 2, 10, seed=40, out_of_place=True).on_gpu()
    c.nt = c.nt[:, :3].contiguous()
    c.run()
    assert c.err.item() == pa.ERRBIT_SEQ_TOO_LONG and (c.nl == 0).all() and (c.kept == -1).all()
    c = Case([100, 90], 2, 64, 16, "f16", 64, 2, 10, seed=40, out_of_place=True).on_gpu()
    c.nt[1, 0] = -1
    c.run()
    assert c.err.item() == pa.ERRBIT_BAD_BLOCK and c.nl.tolist() == [64, 0]


def test_two_evictions_at_once_with_a_workspace_each():
    a = Case([3000, 90], 2, 64, 16, "f16", 200, 2, 30, seed=43, out_of_place=True).on_gpu()
    b = Case([900] * 6, 4, 128, 16, "int4", 640, 2, 30, seed=44, out_of_place=True).on_gpu()
    wants = a.want(), b.want()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(pa.pa_evict_workspace_size(len(c.lens), c.Hkv, c.bt.shape[1] * c.bs, c.budget), dtype=torch.uint8,
                      device="cuda") for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s, w in zip((a, b), streams, ws):
            pa.pa_evict(c.k, c.v, c.wd, c.bt, c.sl, c.nl, c.budget, c.kv, num_sink=c.sink, num_recent=c.recent,
                        new_block_tables=c.nt, kept=c.kept, workspace=w, stream=s)
    torch.cuda.synchronize()
    for c, want in zip((a, b), wants):
        c.check(want)


@pytest.mark.parametrize("D,kv", [(24, "f16"), (80, "bf16"), (256, "f32"), (16, "fp8_e4m3")])
@pytest.mark.parametrize("out_of_place", [False, True])
def test_other_head_dims(D, kv, out_of_place):
    c = Case([150, 90], 3, D, 8, kv, 60, 2, 20, seed=45, out_of_place=out_of_place)
    c.on_gpu().run().check()


def test_pools_of_more_than_four_gigabytes():
    """Rows whose byte offsets pass 32 bits."""
    NB, bs, Hkv, D = 70000, 16, 16, 128                # 4.6 GB per pool
    k = torch.zeros(NB, bs, Hkv, D, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    w = torch.zeros(NB, Hkv, bs, device="cuda")
    bt = torch.arange(NB - 1, NB - 5, -1, dtype=torch.int32, device="cuda").view(1, 4)
    pos = torch.arange(64, device="cuda")
    blk, off = bt[0].long()[pos // bs], pos % bs
    for h in range(Hkv):
        k[blk, off, h] = (pos[:, None] + 100 * h).half()
        v[blk, off, h] = -(pos[:, None] + 100 * h).half()
        w[blk, h, off] = ((pos * 37 + h) % 64).float()
    sl = torch.tensor([64], dtype=torch.int32, device="cuda")
    kept = torch.empty(1, Hkv, 20, dtype=torch.int32, device="cuda")
    score = [[float((t * 37 + h) % 64) for t in range(64)] for h in range(Hkv)]
    pa.pa_evict(k, v, w, bt, sl, sl, 20, num_sink=1, num_recent=4, kept=kept)
    for h in range(Hkv):
        src = _evict.kept_positions(score[h], 20, 1, 4)
        assert kept[0, h].tolist() == src
        for name, sign in ((k, 1), (v, -1)):
            assert torch.equal(name[blk[:20], off[:20], h, 0], sign * (torch.tensor(src, device="cuda") + 100 * h).half())
