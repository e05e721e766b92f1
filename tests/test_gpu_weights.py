"""pa_decode_weights against the formulas in 64 bits, for every cache type;
decode steps with eviction between them, as a server runs them."""
import numpy as np
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _evict
import _int4
from test_gpu_guards import guarded_like, guards_intact

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
OUT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
# rounding of a probability as operand of the second product
PROB = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8, "int4": 2.0 ** -11, "fp8_e4m3": 2.0 ** -11,
        "fp8_e5m2": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa.build()


class Case:
    def __init__(self, lens, Hq, Hkv, D, bs, kv, qd, seed, fresh=None, q_mult=1.0, k_mult=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.bs, self.kv, self.qd, self.fresh = list(lens), bs, kv, qd, fresh
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.tables, self.NB, used = _int4.tables_for(rng, lens, bs)
        x = [rng.standard_normal((self.NB, bs, Hkv, D)) * m for m in (k_mult, 1.0)]
        self.ks, self.vs = 1.0, 1.0
        if kv == "int4":
            self.raw = [_int4.poison(_int4.pack(*_int4.encode(a)), used) for a in x]
            self.val = [_int4.values(p) for p in self.raw]
            self.pool = [torch.from_numpy(p) for p in self.raw]
        else:
            f8 = {"fp8_e4m3": torch.float8_e4m3fn, "fp8_e5m2": torch.float8_e5m2}.get(kv)
            if f8:
                self.ks, self.vs = 0.0125, 0.05
            self.pool = [(torch.from_numpy(a) / s).to(f8 or DT[kv]) for a, s in zip(x, (self.ks, self.vs))]
            v = [p.double().numpy() * np.float32(s).astype(np.float64) for p, s in zip(self.pool, (self.ks, self.vs))]
            self.val = [(a, np.abs(a)) for a in v]
            for p in self.pool:
                nan = torch.full_like(p.float(), float("nan")).to(p.dtype)
                p.copy_(torch.where(torch.from_numpy(used)[:, :, None, None], p.float(), nan.float()).to(p.dtype))
            if kv == "fp8_e4m3":
                self.pool = [p.view(torch.uint8) for p in self.pool]
        self.q = torch.from_numpy(rng.standard_normal((len(lens), Hq, D)) * q_mult).to(DT[qd])
        self.w = np.abs(rng.standard_normal((self.NB, Hkv, bs))).astype(np.float32)
        self.w[~used[:, None, :].repeat(Hkv, 1)] = np.nan
        for i, L in enumerate(self.lens):                      # what a former owner left in fresh slots
            for t in range(max(0, L - (1 if fresh is None else min(fresh[i], L))), L):
                self.w[self.tables[i][t // bs], :, t % bs] = np.nan
        self.scale = 1 / np.sqrt(D) / max(1.0, q_mult * k_mult)

    def want(self):
        """(out, its bound, weights, their bound) in float64."""
        (kv, ka), (vv, va) = ((a.reshape(-1, self.Hkv, self.D) for a in p) for p in self.val)
        G = self.Hq // self.Hkv
        q = self.q.double().numpy()
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        w, wt = self.w.astype(np.float64), np.zeros(self.w.shape)
        for i, L in enumerate(self.lens):
            pos = np.arange(L)
            blk, off = self.tables[i][pos // self.bs].astype(np.int64), pos % self.bs
            sl = blk * self.bs + off
            new = pos >= L - (1 if self.fresh is None else max(0, min(self.fresh[i], L)))
            for g in range(self.Hkv):
                gain, gt = np.zeros(L), np.zeros(L)
                for h in range(g * G, (g + 1) * G):
                    if L == 0:
                        continue
                    s = kv[sl, g] @ q[i, h] * self.scale
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    # scores: D products in f32; a probability moves by twice that (numerator and sum), and
                    # 2^-18 for exp2, the sums over tokens and the division
                    rel = 2 * (self.D + 2) * 2.0 ** -23 * (ka[sl, g] @ np.abs(q[i, h])).max() * self.scale + 2.0 ** -18
                    gain, gt = gain + p, gt + rel * p
                    out[i, h] = p @ vv[sl, g]
                    tol[i, h] = (PROB[self.kv] + rel) * (p @ va[sl, g])
                old = np.where(new, 0.0, w[blk, g, off])
                w[blk, g, off] = old + gain
                # f32 additions of the group's heads, and one to the old sum
                wt[blk, g, off] = gt + (G + 1) * 2.0 ** -24 * (np.abs(old) + gain) + 2.0 ** -120
        return out, tol + OUT[self.qd] * np.abs(out) + 2.0 ** -25, w, wt

    def on_gpu(self):
        self.k, self.v = (p.cuda().contiguous() for p in self.pool)
        self.wd, self.bt = torch.from_numpy(self.w).cuda(), torch.from_numpy(self.tables).cuda()
        self.sl, self.qg = torch.tensor(self.lens, dtype=torch.int32).cuda(), self.q.cuda()
        self.fr = None if self.fresh is None else torch.tensor(self.fresh, dtype=torch.int32).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self

    def run(self, out=None, **kw):
        out = torch.full_like(self.qg, float("nan")) if out is None else out
        pa.pa_decode_weights(out, self.wd, self.qg, self.k, self.v, self.bt, self.sl, self.scale, self.kv,
                             fresh=self.fr, k_scale=self.ks, v_scale=self.vs, err_flag=self.err, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, want=None):
        o, ot, w, wt = want or self.want()
        g = out.double().cpu().numpy()
        assert np.isfinite(g).all()
        assert (np.abs(g - o) <= ot).all(), np.max(np.abs(g - o) - ot)
        got = self.wd.cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(w))
        touched = ~np.isnan(w)
        off = np.abs(got - w)[touched] - wt[touched]
        assert (off <= 0).all(), f"{(off > 0).sum()} weights beyond the bound, worst {off.max():.3g}"


CASES = [
    # lens, Hq, Hkv, D, bs, cache, queries
    ([1], 1, 1, 64, 8, "f16", "f16"),
    ([5, 16, 17, 40], 4, 2, 64, 16, "f32", "f32"),
    ([300, 17, 0, 900, 5, 128], 28, 4, 128, 16, "f16", "f16"),
    ([777, 64, 1, 2049], 32, 8, 128, 32, "bf16", "bf16"),
    ([333, 65], 40, 2, 128, 128, "bf16", "bf16"),
    ([129, 31, 200], 6, 3, 64, 64, "bf16", "bf16"),
    ([300, 17, 0, 900, 5, 128], 28, 4, 128, 16, "int4", "f16"),
    ([250, 31, 33], 7, 1, 128, 8, "int4", "bf16"),
    ([1000, 129, 64, 65], 16, 2, 64, 32, "int4", "bf16"),
    ([500, 70], 24, 1, 128, 16, "int4", "f16"),
    ([140, 33, 600], 8, 2, 128, 16, "fp8_e4m3", "f16"),
    ([140, 33, 600], 32, 2, 128, 32, "fp8_e5m2", "bf16"),
    ([200, 90], 2, 2, 128, 16, "f32", "f32"),
]


@pytest.mark.parametrize("k", range(len(CASES)))
def test_decode_weights(k):
    c = Case(*CASES[k], seed=400 + k).on_gpu()
    c.check(c.run())
    assert c.err.item() == 0


@pytest.mark.parametrize("kv,qd", [("f16", "f16"), ("int4", "bf16"), ("f32", "f32")])
def test_fresh_tokens_start_from_zero(kv, qd):
    c = Case([100, 64, 17, 5, 0], 8, 2, 64, 16, kv, qd, seed=41, fresh=[100, 3, 0, 9, 2]).on_gpu()
    c.check(c.run())


@pytest.mark.parametrize("kv", ["f16", "int4"])
def test_a_long_sequence_and_many_short_ones(kv):
    c = Case([30011, 20], 8, 2, 128, 32, kv, "f16", seed=42).on_gpu()
    c.check(c.run())
    rng = np.random.default_rng(43)
    c = Case(rng.integers(0, 80, 500), 4, 2, 64, 16, kv, "f16", seed=44).on_gpu()
    c.check(c.run())


@pytest.mark.parametrize("kv", ["f16", "int4"])
def test_steep_softmax(kv):
    """Scores tens apart: most weights are nothing, the sum of each head's is still 1."""
    c = Case([500, 64], 8, 2, 128, 16, kv, "f16", seed=45, q_mult=20.0)
    c.scale *= 20
    c.on_gpu()
    c.check(c.run())


def test_output_equals_decode():
    for kv, qd in (("f16", "f16"), ("bf16", "bf16"), ("int4", "bf16"), ("f32", "f32")):
        c = Case([300, 17, 900], 8, 2, 128, 16, kv, qd, seed=46).on_gpu()
        ref = torch.empty_like(c.qg)
        pa.pa_decode(ref, c.qg, c.k, c.v, c.bt, c.sl, c.scale, kv)
        assert torch.equal(c.run(), ref)


@pytest.mark.parametrize("kv", ["f16", "int4"])
def test_guards_repeats_and_a_garbage_workspace(kv):
    c = Case([300, 17, 900], 8, 2, 128, 16, kv, "f16", seed=47).on_gpu()
    w0 = c.wd.clone()
    ws = torch.full((pa.pa_decode_weights_workspace_size(3, 8, c.bt.shape[1] * 16, 128),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    wb, ws = guarded_like(ws)
    pb, c.wd = guarded_like(c.wd)
    ob, out = guarded_like(torch.zeros_like(c.qg))
    c.run(out, workspace=ws)
    c.check(out)
    first = c.wd.clone()
    for _ in range(2):
        c.wd.copy_(w0)
        c.run(out, workspace=ws)
        assert torch.equal(c.wd.view(torch.int32), first.view(torch.int32))
    assert guards_intact(wb) and guards_intact(pb) and guards_intact(ob)


@pytest.mark.parametrize("kv", ["f16", "int4"])
def test_graph_replay_adds_once_per_replay(kv):
    c = Case([300, 17], 8, 2, 128, 16, kv, "f16", seed=48).on_gpu()
    ws = torch.empty(pa.pa_decode_weights_workspace_size(2, 8, c.bt.shape[1] * 16, 128), dtype=torch.uint8, device="cuda")
    w0 = c.wd.clone()
    out = c.run(workspace=ws)
    once = c.wd.clone()
    c.run(workspace=ws)
    twice = c.wd.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_weights(out, c.wd, c.qg, c.k, c.v, c.bt, c.sl, c.scale, c.kv, workspace=ws)
    c.wd.copy_(w0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.wd.view(torch.int32), once.view(torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.wd.view(torch.int32), twice.view(torch.int32))
    s = torch.cuda.Stream()
    c.wd.copy_(w0)
    s.wait_stream(torch.cuda.current_stream())
    c.run(workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(c.wd.view(torch.int32), once.view(torch.int32))


@pytest.mark.parametrize("kv", ["f16", "int4"])
def test_bad_blocks_are_left_out(kv):
    c = Case([100, 60, 40], 8, 2, 64, 16, kv, "f16", seed=49)
    keep = c.tables.copy()
    c.tables[1, 2] = c.NB + 3
    c.on_gpu()
    out = c.run()
    assert c.err.item() == pa.ERRBIT_BAD_BLOCK
    c.tables = keep
    o, ot, w, wt = c.want()
    got = c.wd.cpu().numpy()
    lost = keep[1, 2]
    assert np.array_equal(got[lost].view(np.uint32), c.w[lost].view(np.uint32))      # untouched
    for i in (0, 2):
        assert (np.abs(out[i].double().cpu().numpy() - o[i]) <= ot[i]).all()
        for j in range(-(-c.lens[i] // 16)):
            b = keep[i, j]
            ok = ~np.isnan(w[b])
            assert (np.abs(got[b] - w[b])[ok] <= wt[b][ok]).all()


@pytest.mark.parametrize("kv", ["int4", "f16"])
def test_decode_and_evict_as_a_server_runs_them(kv):
    """Prompts are written, decode steps write, attend and add weights, and every time a sequence passes its budget by
    a block it is brought down to it: outputs, weights and kept tokens of every step against the definitions."""
    rng = np.random.default_rng(50)
    B, Hq, Hkv, D, bs, budget, sink, recent = 2, 8, 2, 64, 16, 64, 2, 12
    lens = [70, 9]
    MB = 8
    tables = rng.permutation(B * MB + 2)[:B * MB].reshape(B, MB).astype(np.int32)
    NB = B * MB + 2
    if kv == "int4":
        k, v = pa.alloc_int4_cache(NB, bs, Hkv, D), pa.alloc_int4_cache(NB, bs, Hkv, D)
    else:
        k = torch.zeros(NB, bs, Hkv, D, dtype=torch.float16, device="cuda")
        v = torch.zeros_like(k)
    wd = torch.full((NB, Hkv, bs), float("nan"), device="cuda")
    bt = torch.from_numpy(tables).cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = torch.empty(B, Hkv, budget, dtype=torch.int32, device="cuda")
    # the model of the cache: per sequence and head a list of (k, v, weight)
    rows = [[[] for _ in range(Hkv)] for _ in range(B)]

    def slot(i, t):
        return int(tables[i][t // bs]) * bs + t % bs

    def write(tok):                                   # [(sequence, position)]
        x = [(rng.standard_normal((len(tok), Hkv, D))).astype(np.float16) for _ in range(2)]
        s = torch.tensor([slot(i, t) for i, t in tok])
        pa.pa_reshape_and_cache(k, v, torch.from_numpy(x[0]).cuda(), torch.from_numpy(x[1]).cuda(), s.cuda(),
                                kv if kv == "int4" else None, err_flag=err)
        held = [_int4.decode(*_int4.encode(a)) if kv == "int4" else a.astype(np.float64) for a in x]
        for n, (i, _) in enumerate(tok):
            for g in range(Hkv):
                rows[i][g].append([held[0][n, g], held[1][n, g], 0.0])

    write([(i, t) for i in range(B) for t in range(lens[i])])
    fresh = torch.tensor(lens, dtype=torch.int32, device="cuda")
    evictions = 0
    for step in range(60):
        if step:
            write([(i, lens[i]) for i in range(B)])
            lens = [L + 1 for L in lens]
            sl += 1
        q = torch.from_numpy(rng.standard_normal((B, Hq, D))).half()
        out = torch.empty_like(q, device="cuda")
        pa.pa_decode_weights(out, wd, q.cuda(), k, v, bt, sl, 0.125, kv, fresh=fresh if step == 0 else None,
                             err_flag=err)
        got = out.double().cpu().numpy()
        for i in range(B):
            for h in range(Hq):
                r = rows[i][h // (Hq // Hkv)]
                K, V = np.stack([a[0] for a in r]), np.stack([a[1] for a in r])
                s = K @ q[i, h].double().numpy() * 0.125
                p = np.exp(s - s.max())
                p /= p.sum()
                want = p @ V
                # 2^-11 each for the output, the probabilities and, on the terms of a 4-bit value (within 6 of 0), their sum
                assert (np.abs(got[i, h] - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -10 * 6).all()
                for a, x in zip(r, p):
                    a[2] += x
        if max(lens) >= budget + bs:
            evictions += 1
            # the sums that decide are the kernels' own: they are checked, then taken over
            w = wd.cpu().numpy()
            for i in range(B):
                for g in range(Hkv):
                    for t, a in enumerate(rows[i][g]):
                        mine = float(w[tables[i][t // bs], g, t % bs])
                        assert abs(mine - a[2]) <= 1e-4 * a[2] + 1e-12
                        a[2] = mine
            pa.pa_evict(k, v, wd, bt, sl, sl, budget, kv, num_sink=sink, num_recent=recent, kept=kept, err_flag=err)
            for i in range(B):
                for g in range(Hkv):
                    src = _evict.kept_positions([a[2] for a in rows[i][g]], budget, sink, recent)
                    assert kept[i, g].tolist()[:len(src)] == src
                    rows[i][g] = [rows[i][g][t] for t in src]
            lens = [min(L, budget) for L in lens]
            assert sl.tolist() == lens
    assert evictions >= 3 and err.item() == 0


def test_manager_gives_back_what_eviction_frees():
    """The host manager's tables through prompts, decode steps and evictions: blocks that a shrink released are taken
    and overwritten by another request, and the evicted one still attends exactly its kept rows."""
    from paged_kv_cache_69_gb300 import block_manager as hbm
    rng = np.random.default_rng(51)
    bs, nb, Hkv, D, Hq, budget, maxb = 16, 24, 2, 64, 4, 48, 16
    m = hbm.HostBlockManager(nb, bs, rng.permutation(nb).tolist())
    k = torch.zeros(nb, bs, Hkv, D, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    wd = torch.zeros(nb, Hkv, bs, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def tokens(req, lo, hi):
        x = [torch.from_numpy(rng.standard_normal((hi - lo, Hkv, D))).half() for _ in range(2)]
        t = m.block_table(req)
        s = torch.tensor([t[p // bs] * bs + p % bs for p in range(lo, hi)])
        pa.pa_reshape_and_cache(k, v, x[0].cuda(), x[1].cuda(), s.cuda(), err_flag=err)
        return x

    m.allocate(0, 150)
    pk, pv = tokens(0, 0, 150)
    q = torch.from_numpy(rng.standard_normal((1, Hq, D))).half().cuda()
    bt = torch.as_tensor(m.block_tables([0], maxb).copy()).cuda()
    sl = torch.tensor([150], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    pa.pa_decode_weights(out, wd, q, k, v, bt, sl, 0.125, fresh=sl.clone(), err_flag=err)
    kept = torch.empty(1, Hkv, budget, dtype=torch.int32, device="cuda")
    free = m.num_free()
    m.shrink(0, budget)
    assert m.num_free() == free + 7
    pa.pa_evict(k, v, wd, bt, sl, sl, budget, num_sink=2, num_recent=8, kept=kept, err_flag=err)
    m.allocate(1, m.num_free() * bs)                       # takes the released blocks
    tokens(1, 0, m.num_tokens(1))
    bt = torch.as_tensor(m.block_tables([0], maxb).copy()).cuda()
    pa.pa_decode(out, q, k, v, bt, sl, 0.125, err_flag=err)
    got = out.double().cpu().numpy()
    src = kept.cpu().numpy()[0]
    assert sl.item() == budget and err.item() == 0
    for h in range(Hq):
        t = src[h // 2]
        assert len(set(t.tolist())) == budget and set(range(2)) <= set(t.tolist()) and t[-8:].tolist() == list(range(142, 150))
        K, V = pk[t, h // 2].double().numpy(), pv[t, h // 2].double().numpy()
        s = K @ q[0, h].double().cpu().numpy() * 0.125
        p = np.exp(s - s.max())
        p /= p.sum()
        # f16 output, probabilities rounded to f16; scores in f32
        assert (np.abs(got[0, h] - p @ V) <= 2.0 ** -11 * np.abs(p @ V) + (2.0 ** -11 + 2.0 ** -17) * (p @ np.abs(V)) + 2.0 ** -25).all()
