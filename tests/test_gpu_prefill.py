"""pa_prefill and pa_prefill_cached against their definition in 64 bits."""
import math

import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _prompt as ref

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


class Case:
    def __init__(self, lens, Hq, Hkv, D, dtype, q_lens=None, seed=0, first=0, behind=0, scale=None):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        q_lens = lens if q_lens is None else q_lens
        self.qs, self.ks = ref.starts(q_lens, first), ref.starts(lens, first)
        self.q = rnd(self.qs[-1] + behind, Hq, D).to(dtype).cuda()
        self.k = (rnd(self.ks[-1] + behind, Hkv, D) + rnd(Hkv, D)).to(dtype).cuda()
        self.v = rnd(self.ks[-1] + behind, Hkv, D).to(dtype).cuda()
        self.scale = D ** -0.5 if scale is None else scale
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.order = g
        self.k_start = None if q_lens is lens else self.dev(self.ks)

    def dev(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def flat(self, **kw):
        out = torch.full_like(self.q, 7.0)
        pa.pa_prefill(out, self.q, self.k, self.v, self.dev(self.qs), self.scale, k_start=self.k_start, err_flag=self.err,
                      **kw)
        return out

    def pools(self, bs):
        return ref.paged(self.k, self.v, self.ks, bs, self.order)

    def cached(self, bs, **kw):
        kc, vc, bt, lens = self.pools(bs)
        out = torch.full_like(self.q, 7.0)
        pa.pa_prefill_cached(out, self.q, kc, vc, bt, lens, self.dev(self.qs), self.scale, err_flag=self.err, **kw)
        return out

    def check(self, out, bits=0):
        want, tol = ref.prompts(self.q, self.k, self.v, self.qs, self.ks, self.scale, 7.0)
        assert self.err.item() == bits
        ref.check(out, want, tol)


EDGE = [1, 0, 2, 127, 128, 129, 255, 256, 257, 300, 3]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (7, 1), (24, 8), (33, 3), (128, 1), (5, 5)])
def test_whole_prompts(dtype, D, Hq, Hkv):
    c = Case(EDGE, Hq, Hkv, D, dtype, seed=Hq + D)
    c.check(c.flat())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
def test_cached_prompts_and_chunks(dtype, D, bs):
    lens = [1, 300, 0, 128, 129, 517, 1000, 64, 16]
    chunk = [1, 300, 0, 1, 129, 130, 333, 17, 5]
    c = Case(lens, 8, 2, D, dtype, q_lens=chunk, seed=bs)
    c.check(c.cached(bs))
    c.check(c.flat())


@pytest.mark.parametrize("B", [33, 70, 200])
def test_many_sequences(B):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 200, (B,), generator=g).tolist()
    chunk = [int(x * torch.rand(1, generator=g)) for x in lens]
    c = Case(lens, 4, 2, 64, BF16, q_lens=chunk, seed=B)
    c.check(c.flat())
    c.check(c.cached(16))


@pytest.mark.parametrize("lens,chunk", [([20000], [1]), ([9000, 300], [40, 3]), ([700], [700]), ([5000, 0, 17], [5, 0, 17])])
def test_few_rows_over_many_keys(lens, chunk):
    """So few items that each is cut into ranges of keys."""
    for D, dtype in ((128, BF16), (64, F16)):
        c = Case(lens, 6, 2, D, dtype, q_lens=chunk, seed=len(lens))
        assert pa.pa_prefill_workspace_size(len(lens), c.q.shape[0], 6, 2, D) > 256
        c.check(c.flat())
        c.check(c.cached(32))


def test_long_prompt():
    c = Case([6000], 2, 1, 128, BF16)
    c.check(c.flat())


def test_more_query_tokens_than_keys_gives_zeros_first():
    c = Case([3, 0, 130], 4, 1, 128, F16, q_lens=[10, 4, 200])
    c.check(c.flat())
    out = c.cached(16)
    c.check(out)
    assert (out[:7] == 0).all() and (out[10:14] == 0).all()


def test_rows_of_no_sequence_are_left():
    c = Case([40, 200], 4, 2, 64, F16, first=9, behind=30)
    out = c.flat()
    c.check(out)
    assert (out[:9] == 7).all() and (out[-30:] == 7).all()


@pytest.mark.parametrize("scale", [-0.3, 0.0, 3.0])
def test_scales(scale):
    c = Case([300, 5], 4, 2, 128, F16, scale=scale)
    c.check(c.flat())


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_growing_scores(dtype):
    """Every chunk's scores pass the reference of those before."""
    c = Case([1500], 2, 1, 64, dtype)
    ramp = torch.linspace(0.1, 8, 1500, device="cuda")[:, None, None]
    c.q[:] = c.q.abs()
    c.k[:] = (c.k.abs() * ramp).to(dtype)
    c.check(c.flat())


def test_one_heavy_key_among_light_ones():
    """f16 weights far below the row's largest still count."""
    c = Case([20000], 1, 1, 64, F16, q_lens=[3])
    c.k[:] = 0
    c.q[:] = 0
    c.q[:, :, 0] = 1
    c.k[:, :, 0] = -12.0                       # weights of 2^-17.3 of the first key's
    c.k[0] = 0
    c.v[:] = 1
    c.v[0] = 0
    c.scale = 1.0
    out = c.flat()
    c.check(out)
    assert (out > 0.1).all()


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("D", [64, 128])
def test_what_a_token_may_not_attend_does_not_reach_it(what, D):
    for dtype, at in ((F16, 70), (BF16, 300), (F16, 299)):
        c = Case([301, 40], 6, 2, D, dtype)
        clean_k, clean_v = c.k.clone(), c.v.clone()
        before = c.flat()
        c.k[at, 1, 3] = what
        out = c.flat()
        assert torch.equal(out[:at], before[:at]) and torch.equal(out[301:], before[301:])
        assert torch.equal(out[:, :3], before[:, :3])
        c.k.copy_(clean_k)
        c.v[at, 0, 5] = what
        for out in (c.flat(), c.cached(16)):
            hit = torch.zeros_like(out, dtype=torch.bool)
            hit[at:301, :3, 5] = True
            assert torch.equal(out[~hit], before[~hit])
            assert not torch.isfinite(out[hit]).any()
            assert out[hit].isnan().all() if math.isnan(what) else (out[hit] == what).all()
        c.v[at - 3, 0, 5] = -what                                     # opposite infinities
        out = c.flat()
        assert out[at:301, :3, 5].isnan().all() and torch.equal(out[:at - 3], before[:at - 3])
        c.v.copy_(clean_v)


def test_scores_of_minus_infinity():
    c = Case([200, 10], 2, 1, 64, BF16)
    c.q[:] = c.q.abs() + 0.5
    c.k[:50] = -math.inf
    out = c.flat()
    assert (out[:50] == 0).all()
    c.check(out)


def test_bad_tables_lengths_and_offsets():
    c = Case([300, 200, 100], 4, 2, 64, F16, q_lens=[30, 200, 100])
    kc, vc, bt, lens = c.pools(16)
    qs = c.dev(c.qs)
    call = lambda bt, lens, qs: pa.pa_prefill_cached(  # noqa: E731
        torch.full_like(c.q, 7.0), c.q, kc, vc, bt, lens, qs, c.scale, err_flag=c.err)
    want, tol = ref.prompts(c.q, c.k, c.v, c.qs, c.ks, c.scale, 7.0)
    # a block outside the pool: its keys are left out, the other sequences are as they were
    b2 = bt.clone()
    b2[1, 3] = kc.shape[0]
    out = call(b2, lens, qs)
    assert c.err.item() == pa.ERRBIT_BAD_BLOCK
    ref.check(out[:30], want[:30], tol[:30])
    ref.check(out[230:], want[230:], tol[230:])
    keep = torch.cat([torch.arange(48), torch.arange(64, 200)]).cuda()
    o, t = ref.attend(c.q[30 + 64:230], c.k[300:500][keep], c.v[300:500][keep], c.scale,
                      torch.arange(48, 184, device="cuda"))
    ref.check(out[94:230], o, t)
    # a sequence longer than its table
    c.err.zero_()
    l2 = lens.clone()
    l2[0] = bt.shape[1] * 16 + 1
    out = call(bt, l2, qs)
    assert c.err.item() == pa.ERRBIT_SEQ_TOO_LONG and (out[:30] == 7).all()
    ref.check(out[30:], want[30:], tol[30:])
    # offsets that decrease, or leave the rows
    for bad in ([0, 30, 10, 330], [0, 30, 230, 331], [-1, 30, 230, 330]):
        c.err.zero_()
        out = call(bt, lens, c.dev(bad))
        assert c.err.item() == pa.ERRBIT_BAD_QUERY
    c.err.zero_()
    pa.pa_prefill(out, c.q, c.k, c.v, qs, c.scale, k_start=c.dev([0, 300, 500, 601]), err_flag=c.err)
    assert c.err.item() == pa.ERRBIT_BAD_QUERY


def test_same_bits_again_on_another_stream_and_from_a_graph():
    c = Case([900, 33, 257], 8, 2, 128, BF16)
    once, qs = c.flat(), c.dev(c.qs)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.full_like(c.q, 7.0)
    pa.pa_prefill(out, c.q, c.k, c.v, qs, c.scale, err_flag=c.err, stream=st)
    st.synchronize()
    assert torch.equal(out, once)
    ws = torch.empty(pa.pa_prefill_workspace_size(3, 1190, 8, 2, 128), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_prefill(out, c.q, c.k, c.v, qs, c.scale, workspace=ws, err_flag=c.err)
    out.fill_(7.0)
    graph.replay()
    assert torch.equal(out, once)
    # other lengths and values under the same graph
    other = Case([1, 1000, 100], 8, 2, 128, BF16, seed=5, behind=89)
    for a, b in ((c.q, other.q), (c.k, other.k), (c.v, other.v)):
        a.copy_(b)
    qs.copy_(c.dev(other.qs))
    out.fill_(7.0)
    graph.replay()
    other.check(out)


def test_two_calls_at_once():
    a, b = Case([700, 3], 8, 2, 128, F16, seed=1), Case([2000], 4, 4, 64, BF16, seed=2)
    wa, wb = a.flat(), b.flat()
    qa, qb = a.dev(a.qs), b.dev(b.qs)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        oa, ob = torch.empty_like(a.q), torch.empty_like(b.q)
        torch.cuda.synchronize()
        pa.pa_prefill(oa, a.q, a.k, a.v, qa, a.scale, stream=s1)
        pa.pa_prefill(ob, b.q, b.k, b.v, qb, b.scale, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_pool_past_4_gb():
    """Rows whose byte offsets pass 32 bits."""
    bs, Hkv, D = 64, 8, 128
    NB = (5 << 30) // (bs * Hkv * D * 2)
    kc = torch.empty(NB, bs, Hkv, D, dtype=F16, device="cuda")
    vc = torch.empty_like(kc)
    c = Case([200], 8, Hkv, D, F16, q_lens=[70])
    bt = torch.tensor([[NB - 1, 0, NB // 2, NB - 3]], dtype=torch.int32, device="cuda")
    for t in range(0, 200, bs):
        n = min(bs, 200 - t)
        kc[bt[0, t // bs], :n], vc[bt[0, t // bs], :n] = c.k[t:t + n], c.v[t:t + n]
    vc[bt[0, 3], 8:] = math.nan
    out = torch.empty_like(c.q)
    pa.pa_prefill_cached(out, c.q, kc, vc, bt, c.dev([200]), c.dev([0, 70]), c.scale, err_flag=c.err)
    c.check(out)


def test_agrees_with_pa_attention():
    c = Case([900, 80], 8, 2, 128, F16, q_lens=[7, 3])
    kc, vc, bt, lens = c.pools(16)
    a, b = torch.empty_like(c.q), torch.empty_like(c.q)
    pa.pa_prefill_cached(a, c.q, kc, vc, bt, lens, c.dev(c.qs), c.scale, err_flag=c.err)
    pa.pa_attention(b, c.q, kc, vc, bt, lens, c.dev(c.qs), c.scale, 7, err_flag=c.err)
    want, tol = ref.prompts(c.q, c.k, c.v, c.qs, c.ks, c.scale, 7.0)
    c.check(a)
    ref.check(b, a.double(), 2 * tol)


def test_more_sequences_than_the_scheduler_keeps():
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 40, (1500,), generator=g).tolist()
    lens[1400] = 700
    c = Case(lens, 2, 1, 64, F16, seed=1)
    c.check(c.flat())


def test_lengths_of_many_levels():
    """128 heads to a KV head: an item is two tokens, its levels are counted by steps."""
    c = Case([1, 4097, 3000, 17], 128, 1, 64, BF16, q_lens=[1, 2300, 5, 17])
    c.check(c.flat())


@pytest.mark.parametrize("Hkv", [1, 3, 16])
def test_items_about_a_round(Hkv):
    """Just under, at and over whole rounds of items, whose rest is cut."""
    for n in (36, 2700, 152 * 36 // Hkv, 152 * 36 // Hkv + 1, 160 * 36 // Hkv, 300 * 36 // Hkv):
        c = Case([n + 3000], 7 * Hkv, Hkv, 64, F16, q_lens=[n], seed=n)
        out = c.flat()
        rows = torch.randperm(n, generator=c.order)[:40].sort().values
        o, t = ref.attend(c.q[rows.cuda()], c.k, c.v, c.scale, (rows + 3000).cuda())
        ref.check(out[rows.cuda()], o, t)
        assert c.err.item() == 0


def test_no_keys_at_all():
    c = Case([0, 0], 4, 2, 64, F16, q_lens=[3, 5])
    out = c.flat()
    assert c.k.shape[0] == 0 and (out == 0).all() and c.err.item() == 0


@pytest.mark.parametrize("k", [5, 20, 40, 51, 76, 79, 100, 130])
def test_spans_of_cut_items(k):
    """2 k items, every row of them: cut into spans that end inside an item and start in the one before."""
    n = 36 * k - 5
    c = Case([n + 2500], 14, 2, 64, BF16, q_lens=[n], seed=k)
    want, tol = ref.attend(c.q, c.k, c.v, c.scale, torch.arange(2500, 2500 + n, device="cuda"))
    for out in (c.flat(), c.cached(64)):
        ref.check(out, want, tol)
    assert c.err.item() == 0


@pytest.mark.parametrize("lens,chunk", [([6000, 900, 3000], [1500, 700, 36]), ([4000, 4000, 200, 100], [1300, 900, 200, 100]),
                                        ([2000] * 9, [300] * 9), ([5000, 60, 50, 40], [700, 60, 50, 40])])
def test_spans_of_unequal_items(lens, chunk):
    c = Case(lens, 14, 2, 128, F16, q_lens=chunk, seed=len(lens))
    c.check(c.flat())
    c.check(c.cached(16))
