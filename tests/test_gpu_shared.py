"""pa_decode_shared against its definition in 64 bits, and beside pa_decode."""
import math

import pytest
import torch

import paged_kv_cache_69_gb300 as pa
from paged_kv_cache_69_gb300.block_manager import HostBlockManager

import _prompt as ref

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


class Case:
    """groups: (members, shared tokens, own tokens of each member)."""

    def __init__(self, groups, Hq, Hkv, D, dtype, bs=16, seed=0, spare=2, scale=None):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.bs, self.scale = bs, D ** -0.5 if scale is None else scale
        need = sum(P // bs + sum(-(-(P % bs + o) // bs) for o in own) for P, own in groups)
        NB = need + spare
        perm = iter(torch.randperm(NB, generator=g).tolist())
        rows, lens, starts, prefix = [], [], [0], []
        for P, own in groups:
            common = [next(perm) for _ in range(P // bs)]
            for o in own:
                rows.append(common + [next(perm) for _ in range(-(-(P % bs + o) // bs))])
                lens.append(P + o)
            starts.append(len(lens))
            prefix.append(P)
        MB = max([len(r) for r in rows] + [0]) + 1
        fill = [NB + 7, -1] * MB
        self.tables = self.dev([r + fill[:MB - len(r)] for r in rows])
        self.lens, self.starts, self.prefix = self.dev(lens), self.dev(starts), self.dev(prefix)
        self.k = torch.full((NB, bs, Hkv, D), math.nan, dtype=dtype, device="cuda")
        self.v = self.k.clone()
        mean = rnd(Hkv, D)
        for i, (r, L) in enumerate(zip(rows, lens)):
            first = 0 if i in starts else (prefix[sum(s <= i for s in starts) - 1] // bs * bs)
            pos = torch.arange(first, L)
            if pos.numel():
                blk, off = torch.tensor(r)[pos // bs].cuda(), (pos % bs).cuda()
                self.k[blk, off] = (rnd(pos.numel(), Hkv, D) + mean).to(dtype).cuda()
                self.v[blk, off] = rnd(pos.numel(), Hkv, D).to(dtype).cuda()
        self.q = rnd(len(lens), Hq, D).to(dtype).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def dev(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def call(self, **kw):
        out = torch.full_like(self.q, 7.0)
        kw.setdefault("err_flag", self.err)
        pa.pa_decode_shared(out, self.q, self.k, self.v, self.tables, self.lens, self.starts, self.prefix, self.scale, **kw)
        return out

    def want(self):
        out = torch.zeros(self.q.shape, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        for i, L in enumerate(self.lens.tolist()):
            pos = torch.arange(L, device="cuda")
            blk, off = self.tables[i].long()[pos // self.bs], pos % self.bs
            k, v = self.k[blk, off], self.v[blk, off]
            out[i:i + 1], tol[i:i + 1] = ref.attend(self.q[i:i + 1], k, v, self.scale, self.dev([L - 1]))
            if L and self.q.dtype == F16:
                # the decode kernel's f16 weights have steps of 2^-24 of the row's largest
                tol[i] += L * 2.0 ** -25 * float(v.double().abs().max())
        return out, tol

    def check(self, out, bits=0):
        assert self.err.item() == bits
        ref.check(out, *self.want())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (28, 4), (24, 8), (16, 1)])
def test_groups_of_all_kinds(dtype, D, Hq, Hkv):
    # (some share so little that they are left to the decode kernel)
    groups = [(768, [5, 300, 1, 17]), (0, [40, 3]), (64, [9]), (1000, [1, 2, 0, 30, 20, 700]), (48, [1] * 11), (2176, [0, 0]),
              (16, [5, 5]), (256, [3] * 9), (4000, [7])]
    c = Case(groups, Hq, Hkv, D, dtype, seed=Hq)
    c.check(c.call())


@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
def test_block_sizes_and_prefixes_inside_a_block(bs):
    """What lies behind the prefix's last whole block is each sequence's own."""
    c = Case([(bs * 40 + 3, [5, 40, 1] * 5), (bs - 1, [1, 2] * 6), (bs * 20 + 256, [0, 9] * 4), (bs * 7, [2] * 4)], 8, 2, 128, F16,
             bs=bs)
    c.check(c.call())


@pytest.mark.parametrize("members", [1, 2, 31, 32, 33, 64, 65, 200])
def test_members(members):
    c = Case([(700, [3 + i % 50 for i in range(members)])], 8, 2, 64, BF16, seed=members)
    c.check(c.call())


def test_many_groups():
    g = torch.Generator().manual_seed(3)
    r = lambda a, b: int(torch.randint(a, b + 1, (1,), generator=g))  # noqa: E731
    c = Case([(r(0, 400), [r(0, 60) for _ in range(r(1, 6))]) for _ in range(80)], 14, 2, 128, F16)
    c.check(c.call())


def test_long_prefix_and_long_tails():
    c = Case([(20000, [1, 9000, 30, 5000]), (130, [12000] * 3)], 12, 2, 128, BF16)
    c.check(c.call())


def test_no_group_and_sequences_in_none():
    c = Case([(900, [5, 6, 7, 8]), (2100, [9, 10])], 16, 2, 64, F16)
    want = c.want()
    for starts, prefix, bits in (([0], [], 0), ([0, 4], [900], 0), ([4, 6], [2100], 0),
                                 ([0, 0, 4, 4, 6], [50, 900, 9, 2100], 0), ([0, 2, 1, 6], [900, 800, 0], pa.ERRBIT_BAD_QUERY),
                                 ([0, 4, 9], [900, 2100], pa.ERRBIT_BAD_QUERY), ([-1, 4, 6], [900, 2100], pa.ERRBIT_BAD_QUERY),
                                 ([0, 4, 6], [900, -5], 0), ([0, 4, 6], [-2 ** 31, 700], 0)):
        c.starts, c.prefix = c.dev(starts), c.dev(prefix)
        c.err.zero_()
        out = c.call()
        assert c.err.item() == bits
        ref.check(out, *want)


def test_lengths_that_do_not_fit():
    for shared in (320, 960):
        c = Case([(shared, [5, 6, 7, 8]), (200, [9, 10])], 16, 2, 64, F16)
        want, tol = c.want()
        c.lens[1], c.lens[5] = shared - 20, c.tables.shape[1] * 16 + 1
        out = c.call()
        assert c.err.item() == pa.ERRBIT_SEQ_TOO_LONG
        assert (out[1] == 7).all() and (out[5] == 7).all()
        keep = torch.tensor([0, 2, 3, 4], device="cuda")
        ref.check(out[keep], want[keep], tol[keep])


def test_blocks_outside_the_pool_are_left_out():
    c = Case([(960, [5, 60, 7, 8]), (200, [9, 10])], 16, 2, 64, F16)
    want, tol = c.want()
    own = c.tables.clone()
    c.tables[1, 61] = -3                                   # tokens 976..991 of sequence 1
    out = c.call()
    assert c.err.item() == pa.ERRBIT_BAD_BLOCK
    keep = torch.tensor([0, 2, 3, 4, 5], device="cuda")
    ref.check(out[keep], want[keep], tol[keep])
    c.err.zero_()
    c.tables.copy_(own)
    c.tables[0, 2] = c.k.shape[0]                          # tokens 32..47 of the shared prefix
    out = c.call()
    assert c.err.item() == pa.ERRBIT_BAD_BLOCK
    ref.check(out[4:], want[4:], tol[4:])
    for i in range(4):
        L = int(c.lens[i])
        pos = torch.cat([torch.arange(32), torch.arange(48, L)]).cuda()
        blk, off = own[i].long()[pos // 16], pos % 16
        o, t = ref.attend(c.q[i:i + 1], c.k[blk, off], c.v[blk, off], c.scale, c.dev([L]))
        ref.check(out[i:i + 1], o, t + L * 2.0 ** -22)


@pytest.mark.parametrize("scale", [-0.4, 0.0, 2.0])
def test_scales(scale):
    c = Case([(900, [5, 60, 7, 8]), (100, [9, 10])], 16, 2, 128, F16, scale=scale)
    c.check(c.call())


def test_nan_and_infinity():
    """In the prefix they reach every member, in a tail only its own sequence."""
    c = Case([(1024, [5, 20, 7, 8])], 8, 1, 64, BF16)
    before = c.call()
    blk, off = int(c.tables[2, 64]), 3
    c.v[blk, off, 0, 9] = math.inf
    out = c.call()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[2, :, 9] = True
    assert torch.equal(out[~hit], before[~hit]) and (out[hit] == math.inf).all()
    c.k[int(c.tables[0, 1]), 4, 0, 0] = math.nan
    assert c.call().isnan().all()


def test_same_bits_again_and_from_a_graph():
    c = Case([(1024, [5, 20, 7, 100]), (300, [50, 60])], 28, 4, 128, F16, spare=60)
    once = c.call()
    assert torch.equal(c.call(), once)
    ws = torch.empty(pa.pa_decode_shared_workspace_size(6, 2, 28, 4, c.tables.shape[1] * 16, 128), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty_like(c.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_shared(out, c.q, c.k, c.v, c.tables, c.lens, c.starts, c.prefix, c.scale, workspace=ws, err_flag=c.err)
    graph.replay()
    assert torch.equal(out, once)
    # other groups, tables and lengths under the same graph
    o = Case([(64, [1]), (600, [30, 40, 5, 6, 7])], 28, 4, 128, F16, seed=9)
    c.k[:o.k.shape[0]], c.v[:o.v.shape[0]] = o.k, o.v
    c.tables.fill_(-1)
    w = min(o.tables.shape[1] - 1, c.tables.shape[1])
    c.tables[:, :w] = o.tables[:, :w]
    for n in ("q", "lens", "starts", "prefix"):
        getattr(c, n).copy_(getattr(o, n))
    out.fill_(7)
    graph.replay()
    o.check(out)
    assert c.err.item() == 0


def test_two_calls_at_once():
    a = Case([(1024, [5, 20, 7, 100])], 28, 4, 128, F16)
    b = Case([(700, [5] * 40)], 8, 2, 64, BF16)
    wa, wb = a.call(), b.call()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        oa, ob = torch.empty_like(a.q), torch.empty_like(b.q)
        torch.cuda.synchronize()
        for c, o, s in ((a, oa, s1), (b, ob, s2)):
            pa.pa_decode_shared(o, c.q, c.k, c.v, c.tables, c.lens, c.starts, c.prefix, c.scale, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_beside_pa_decode():
    c = Case([(0, [900, 80, 1, 0]), (32, [1, 5])], 8, 2, 128, F16)
    out = torch.empty_like(c.q)
    pa.pa_decode(out, c.q, c.k, c.v, c.tables, c.lens, c.scale)
    want, tol = c.want()
    ref.check(c.call(), out.double(), 2 * tol)


def test_a_request_from_prompt_to_shared_decode():
    """The calls as a serving loop makes them: a prompt rotated and cached, attended,
    forked into branches, and two decode steps of all branches, against dense attention
    over the rotated rows."""
    Hq, Hkv, D, bs, n, branches = 8, 2, 64, 16, 603, 6
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g).to(F16).cuda()  # noqa: E731
    table = pa.rope_table(1000, D)
    bm = HostBlockManager(64, bs)
    kc = torch.full((64, bs, Hkv, D), math.nan, dtype=F16, device="cuda")
    vc = kc.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda x, t=torch.int32: torch.tensor(x, dtype=t, device="cuda")  # noqa: E731
    scale = D ** -0.5
    # the prompt
    bm.allocate(0, n)
    tab = bm.block_table(0)
    slots = dev([tab[t // bs] * bs + t % bs for t in range(n)], torch.int64)
    q, k, v = rnd(n, Hq, D), rnd(n, Hkv, D), rnd(n, Hkv, D)
    key = torch.empty_like(k)
    pa.pa_rope_and_cache(kc, vc, q, q, k, v, torch.arange(n, device="cuda"), table, slots, key_out=key, err_flag=err)
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    pa.pa_prefill(out, q, key, v, dev([0, n]), scale, err_flag=err)
    pa.pa_prefill_cached(out2, q, kc, vc, dev([tab]), dev([n]), dev([0, n]), scale, err_flag=err)
    want, tol = ref.attend(q, key, v, scale, torch.arange(n, device="cuda"))
    ref.check(out, want, tol)
    ref.check(out2, want, tol)
    # the branches
    for b in range(1, branches):
        bm.fork(0, b)
    keys, values = [[key] for _ in range(branches)], [[v] for _ in range(branches)]
    for step in range(2):
        new, pairs, _ = bm.append_slots(list(range(branches)))
        if len(pairs):
            pa.pa_copy_blocks(kc, vc, dev(pairs.tolist(), torch.int64), err_flag=err)
        q, k, v = rnd(branches, Hq, D), rnd(branches, Hkv, D), rnd(branches, Hkv, D)
        pos = torch.full((branches,), n + step, device="cuda")
        key = torch.empty_like(k)
        pa.pa_rope_and_cache(kc, vc, q, q, k, v, pos, table, dev(new.tolist(), torch.int64), key_out=key, err_flag=err)
        tabs = [bm.block_table(b) for b in range(branches)]
        lens = dev([n + step + 1] * branches)
        out = torch.empty_like(q)
        pa.pa_decode_shared(out, q, kc, vc, dev(tabs), lens, dev([0, branches]), dev([n]), scale, err_flag=err)
        for b in range(branches):
            keys[b].append(key[b:b + 1])
            values[b].append(v[b:b + 1])
            want, tol = ref.attend(q[b:b + 1], torch.cat(keys[b]), torch.cat(values[b]), scale, dev([n + step]))
            ref.check(out[b:b + 1], want, tol + 700 * 2.0 ** -25 * 5)
    assert err.item() == 0
