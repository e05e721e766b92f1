"""pa_rope_and_cache against its definition in 64 bits, and its quantised pools
against pa_reshape_and_cache of the rotated keys."""
import math

import pytest
import torch

import paged_kv_cache_69_gb300 as pa

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALF = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}         # a rounding, relative
TINY = {F32: 2.0 ** -150, F16: 2.0 ** -25, BF16: 2.0 ** -134}      # and of the smallest numbers


def turn(x, positions, table, sections, interleaved):
    """(rotated x, tolerance) in float64.  The two products and their difference
    are rounded in f32, the result once to x's type."""
    rot = table.shape[1]
    half = rot // 2
    pos = positions.view(-1, x.shape[0])
    axis = [0] * half if sections is None else [a for a, n in enumerate(sections) for _ in range(n)]
    y, tol = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    for i in range(half):
        c, s = (table[pos[axis[i]], k].double()[:, None] for k in (i, half + i))
        i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = x[..., i0].double(), x[..., i1].double()
        for k, (u, w) in ((i0, (a * c, -b * s)), (i1, (b * c, a * s))):
            y[..., k] = u + w
            size = (u.abs() + w.abs()) * (1 + 2.0 ** -20)
            tol[..., k] = size * 2 * 2.0 ** -24 + (y[..., k].abs() + size * 2 * 2.0 ** -24) * HALF[x.dtype] + TINY[x.dtype]
    return y, tol


def agree(got, want, tol):
    g = got.double()
    ok = (g == want) | ((g - want).abs() <= tol) | (g.isnan() & want.isnan())
    assert ok.all(), f"{int((~ok).sum())} of {ok.numel()}: {float(g[~ok][0])} for {float(want[~ok][0])}"


def same(*pairs):
    """Equal bit by bit (NaN among them)."""
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(pairs[::2], pairs[1::2]))


class Case:
    def __init__(self, T, Hq, Hkv, D, dtype, rot=None, sections=None, interleaved=False, bs=16, seed=0, spare=3,
                 positions=5000):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.q = rnd(T, Hq, D).to(dtype).cuda() if Hq else None
        self.key, self.value = rnd(T, Hkv, D).to(dtype).cuda(), rnd(T, Hkv, D).to(dtype).cuda()
        self.table = pa.rope_table(positions, rot or D)
        n = 1 if sections is None else len(sections)
        self.pos = torch.randint(0, positions, (n, T), generator=g).cuda()
        if sections is None:
            self.pos = self.pos[0]
        self.sections, self.interleaved, self.dtype = sections, interleaved, dtype
        self.NB = -(-T // bs) + spare
        self.bs, self.Hkv, self.D = bs, Hkv, D
        self.slots = torch.randperm(self.NB * bs, generator=g)[:T].cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def pools(self, kv=None):
        if kv == "int4":
            k = pa.alloc_int4_cache(self.NB, self.bs, self.Hkv, self.D)
        else:
            t = {"fp8_e4m3": torch.uint8, "fp8_e5m2": torch.uint8}.get(kv, self.dtype)
            k = torch.full((self.NB, self.bs, self.Hkv, self.D), 3, dtype=t, device="cuda")
        return k, k.clone()

    def call(self, k, v, q_out, kv=None, **kw):
        kw.setdefault("err_flag", self.err)
        pa.pa_rope_and_cache(k, v, q_out, self.q, self.key, self.value, self.pos, self.table, self.slots, kv,
                             sections=self.sections, interleaved=self.interleaved, **kw)

    def turned(self, x):
        return turn(x, self.pos, self.table, self.sections, self.interleaved)

    def check(self):
        k, v = self.pools()
        q_out = None if self.q is None else torch.full_like(self.q, 9)
        key_out = torch.full_like(self.key, 9)
        self.call(k, v, q_out, key_out=key_out)
        assert self.err.item() == 0
        if self.q is not None:
            agree(q_out, *self.turned(self.q))
        agree(key_out, *self.turned(self.key))
        kr, vr = self.pools()
        kr.view(-1, self.Hkv, self.D)[self.slots] = key_out
        vr.view(-1, self.Hkv, self.D)[self.slots] = self.value
        assert same(k, kr, v, vr)
        # without the rotated keys, and in place, the same bits
        k2, v2 = self.pools()
        q, key = None if self.q is None else self.q.clone(), self.key.clone()
        pa.pa_rope_and_cache(k2, v2, q, q, key, self.value, self.pos, self.table, self.slots, sections=self.sections,
                             interleaved=self.interleaved, key_out=key, err_flag=self.err)
        assert same(k2, k, v2, v, key, key_out)
        assert q is None or same(q, q_out)
        k3, v3 = self.pools()
        self.call(k3, v3, q_out)
        assert same(k3, k, v3, v)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 4, 2), (7, 28, 4), (65, 5, 1), (1201, 9, 3)])
def test_one_axis(dtype, D, rot, interleaved, T, Hq, Hkv):
    Case(T, Hq, Hkv, D, dtype, rot, interleaved=interleaved, seed=T).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,sections", [(128, [16, 24, 24]), (128, [64, 0]), (128, [0, 64]), (96, [1, 46, 1]),
                                          (64, [9, 7, 5, 11]), (128, [0, 0, 30, 34])])
def test_several_axes(dtype, interleaved, rot, sections):
    for T in (5, 900):
        Case(T, 14, 2, 128, dtype, rot, sections=sections, interleaved=interleaved).check()


def test_keys_and_values_alone():
    Case(33, 0, 4, 128, F16).check()


@pytest.mark.parametrize("kv", ["fp8_e4m3", "fp8_e5m2", "int4"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_quantised_pools_hold_what_a_write_of_the_rotated_key_gives(kv, dtype, D):
    for T, inter in ((3, False), (700, True), (3000, False)):
        c = Case(T, 8, 2, D, dtype, D // 2, interleaved=inter, seed=T)
        c.key[0] *= 1000
        (k, v), (k2, v2) = c.pools(kv), c.pools(kv)
        q_out, key_out = torch.empty_like(c.q), torch.empty_like(c.key)
        c.call(k, v, q_out, kv, key_out=key_out, k_scale=0.03, v_scale=0.02)
        pa.pa_reshape_and_cache(k2, v2, key_out, c.value, c.slots, kv, k_scale=0.03, v_scale=0.02, err_flag=c.err)
        assert c.err.item() == 0 and torch.equal(k, k2) and torch.equal(v, v2)
        agree(key_out, *c.turned(c.key))
        k3, v3 = c.pools(kv)
        c.call(k3, v3, q_out, kv, k_scale=0.03, v_scale=0.02)
        assert torch.equal(k, k3) and torch.equal(v, v3)


@pytest.mark.parametrize("kv", [None, "fp8_e4m3", "int4"])
def test_padding_and_bad_tokens_write_nothing(kv):
    for T in (40, 2000):
        c = Case(T, 8, 2, 128, F16, sections=[32, 32])
        k, v = c.pools(kv)
        q_out, key_out = torch.full_like(c.q, 9), torch.full_like(c.key, 9)
        c.call(k, v, q_out, kv, key_out=key_out)
        skip = {3: (None, -1), 9: (None, c.NB * c.bs), 20: ((0, 5000), None), 21: ((1, -1), None), 30: (None, 1 << 40),
                T - 1: ((1, 1 << 40), None)}
        good = c.slots.clone()
        for t, (p, s) in skip.items():
            if s is not None:
                c.slots[t] = s
            if p is not None:
                c.pos[p[0], t] = p[1]
        k2, v2 = c.pools(kv)
        fresh = c.pools(kv)[0]
        q2, key2 = torch.full_like(c.q, 9), torch.full_like(c.key, 9)
        c.call(k2, v2, q2, kv, key_out=key2)
        assert c.err.item() == pa.ERRBIT_BAD_SLOT | pa.ERRBIT_BAD_POSITION
        at = torch.tensor(sorted(skip), device="cuda")
        q_out[at], key_out[at] = 9, 9
        assert torch.equal(q2, q_out) and torch.equal(key2, key_out)
        if kv != "int4":
            for x in (k, v):
                x.view(-1, 2, 128)[good[at]] = fresh.view(-1, 2, 128)[good[at]]
            assert torch.equal(k2, k) and torch.equal(v2, v)
        else:
            keep = torch.ones(T, dtype=torch.bool, device="cuda")
            keep[at] = False
            want = c.pools(kv)
            pa.pa_reshape_and_cache(*want, key_out[keep], c.value[keep], good[keep], kv)
            assert torch.equal(k2, want[0]) and torch.equal(v2, want[1])
        c.err.zero_()
        c.pos[0, 20], c.pos[1, 21], c.pos[1, T - 1] = 0, 0, 0
        c.slots[9], c.slots[30] = -5, -1
        c.call(k2, v2, q2, kv)
        assert c.err.item() == 0


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_infinities_and_nan_stay_in_their_pair(dtype):
    c = Case(6, 2, 1, 64, dtype)
    c.q[2, 1, 3], c.key[4, 0, 40], c.value[1, 0, 0] = math.inf, math.nan, -math.inf
    c.check()
    k, v = c.pools()
    q_out = torch.empty_like(c.q)
    c.call(k, v, q_out)
    bad = ~torch.isfinite(q_out)
    assert set(map(tuple, torch.nonzero(bad).tolist())) <= {(2, 1, 3), (2, 1, 35)}


def test_no_tokens():
    c = Case(0, 4, 2, 64, F16)
    k, v = c.pools()
    before = k.clone()
    c.call(k, v, torch.empty_like(c.q))
    assert torch.equal(k, before)


def test_stream_and_graph():
    c = Case(64, 28, 4, 128, BF16)
    k, v = c.pools()
    q_out = torch.empty_like(c.q)
    c.call(k, v, q_out)
    torch.cuda.synchronize()
    k2, v2 = c.pools()
    q2 = torch.empty_like(c.q)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.call(k2, v2, q2, stream=st)
    st.synchronize()
    assert torch.equal(k, k2) and torch.equal(v, v2) and torch.equal(q_out, q2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(k2, v2, q2)
    other = Case(64, 28, 4, 128, BF16, seed=4)
    for n in ("q", "key", "value", "pos", "slots"):
        getattr(c, n).copy_(getattr(other, n))
    k2.copy_(other.pools()[0])
    v2.copy_(k2)
    graph.replay()
    k, v = other.pools()
    other.call(k, v, q_out)
    assert torch.equal(k, k2) and torch.equal(v, v2) and torch.equal(q_out, q2)


def test_pool_past_4_gb():
    c = Case(50, 2, 8, 128, F16, spare=0)
    NB = (5 << 30) // (16 * 8 * 128 * 2)
    k = torch.zeros(NB, 16, 8, 128, dtype=F16, device="cuda")
    v = torch.zeros_like(k)
    c.slots += NB * 16 - c.NB * 16
    q_out, key_out = torch.empty_like(c.q), torch.empty_like(c.key)
    c.call(k, v, q_out, key_out=key_out)
    assert torch.equal(k.view(-1, 8, 128)[c.slots], key_out) and torch.equal(v.view(-1, 8, 128)[c.slots], c.value)
    assert int((k != 0).any(-1).any(-1).sum()) == 50


def test_far_positions_come_from_the_table():
    """Angles of far positions are the table's, in 64 bits."""
    t = pa.rope_table(131072, 128)
    p, i = 131071, torch.arange(64, dtype=torch.float64)
    a = p * 10000.0 ** (-2 * i / 128)
    assert (t[p, :64].cpu().double() - a.cos()).abs().max() < 2.0 ** -24
    assert (t[p, 64:].cpu().double() - a.sin()).abs().max() < 2.0 ** -24
