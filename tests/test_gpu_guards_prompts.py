"""Out-of-bounds write checks of the prompt, rotation and shared-prefix calls: every buffer
that they write -- outputs, rotated rows, pools, workspaces of exactly the size asked for and
full of 0xff -- lies between canaries that must be unchanged, and the results are those of
unguarded calls, bit for bit."""
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _prompt as ref
import test_gpu_shared as shared
from test_gpu_guards import guarded_like, guards_intact, same_bits

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def dev(x, t=torch.int32):
    return torch.tensor(x, dtype=t, device="cuda")


def guarded_workspace(nbytes):
    return guarded_like(torch.full((nbytes,), 0xff, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype,D", [(F16, 128), (BF16, 64)])
@pytest.mark.parametrize("n,lens", [([300, 1, 0, 129, 10], [300, 1, 0, 129, 4]), ([40, 3], [9000, 3]), ([700] * 3, [2500] * 3),
                                    ([1], [20000]), ([2], [0])])
def test_prompts(dtype, D, n, lens):
    Hq, Hkv = 14, 2
    g = torch.Generator().manual_seed(sum(n))
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    qs, ks, err = ref.starts(n), ref.starts(lens), dev([0])
    q, k, v = rnd(qs[-1], Hq, D), rnd(ks[-1], Hkv, D), rnd(ks[-1], Hkv, D)
    kc, vc, bt, sl = ref.paged(k, v, ks, 16, g)
    size = pa.pa_prefill_workspace_size(len(n), qs[-1], Hq, Hkv, D)
    for call in (lambda o, w: pa.pa_prefill(o, q, k, v, dev(qs), 0.1, k_start=dev(ks), workspace=w, err_flag=err),
                 lambda o, w: pa.pa_prefill_cached(o, q, kc, vc, bt, sl, dev(qs), 0.1, workspace=w, err_flag=err)):
        own = torch.empty_like(q)
        call(own, None)
        obuf, out = guarded_like(torch.full_like(q, 7))
        wbuf, ws = guarded_workspace(size)
        call(out, ws)
        torch.cuda.synchronize()
        assert guards_intact(obuf) and guards_intact(wbuf)
        assert same_bits(out, own) and err.item() == 0


@pytest.mark.parametrize("dtype,D", [(F16, 128), (BF16, 64)])
@pytest.mark.parametrize("groups", [[(1024, [5, 20, 7, 100]), (300, [50, 60])], [(2048, [1 + i for i in range(70)])],
                                    [(20000, [3])], [(9008, [1, 700])], [(16, [1])] * 40 + [(2100, [9, 8])] * 20])
def test_shared_prefixes(dtype, D, groups):
    c = shared.Case(groups, 14, 2, D, dtype)
    once = c.call()
    obuf, out = guarded_like(torch.full_like(c.q, 7))
    wbuf, ws = guarded_workspace(pa.pa_decode_shared_workspace_size(c.q.shape[0], len(groups), 14, 2, c.tables.shape[1] * c.bs, D))
    pa.pa_decode_shared(out, c.q, c.k, c.v, c.tables, c.lens, c.starts, c.prefix, c.scale, workspace=ws, err_flag=c.err)
    torch.cuda.synchronize()
    assert guards_intact(obuf) and guards_intact(wbuf)
    assert same_bits(out, once) and c.err.item() == 0


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("kv", [None, "fp8_e5m2", "int4"])
@pytest.mark.parametrize("D,rot", [(64, 48), (128, 128)])
@pytest.mark.parametrize("T", [1, 33, 2500])
def test_rotation(dtype, kv, D, rot, T):
    """The pools' first and last slots among those written, padding and bad slots and positions beside them."""
    g = torch.Generator().manual_seed(T + D)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    q, k, v, table, err = rnd(T, 6, D), rnd(T, 2, D), rnd(T, 2, D), pa.rope_table(T, rot), dev([0])
    NB = -(-T // 16) + 1
    slots = torch.randperm(NB * 16 - 2, generator=g)[:T] + 1                          # (no slot twice)
    slots[0], slots[-1] = NB * 16 - 1, 0
    pos = torch.arange(T)
    if T > 1:
        slots[1:4], pos[4:6] = torch.tensor([-1, NB * 16, 2 ** 40]), torch.tensor([T, -1])
    slots, pos = slots.cuda(), pos.cuda()
    width, of = (D // 2 + 4, torch.uint8) if kv == "int4" else (D, torch.uint8 if kv else dtype)
    pool = torch.full((NB, 16, 2, width), 3, dtype=of, device="cuda")
    seven = torch.full_like(q, 7), torch.full_like(k, 7)
    own = [pool.clone(), pool.clone(), seven[0].clone(), seven[1].clone()]
    pairs = [guarded_like(x) for x in own]
    for kc, vc, qo, ko in (own, [view for _, view in pairs]):
        pa.pa_rope_and_cache(kc, vc, qo, q, k, v, pos, table, slots, kv, key_out=ko, err_flag=err)
    torch.cuda.synchronize()
    assert all(guards_intact(buf) for buf, _ in pairs)
    assert all(same_bits(a, view) for a, (_, view) in zip(own, pairs))
    assert err.item() == (pa.ERRBIT_BAD_SLOT | pa.ERRBIT_BAD_POSITION if T > 1 else 0)
    if T > 1:
        assert (own[2][1:6] == 7).all() and (own[3][1:6] == 7).all() and not (own[2][6:] == 7).all(-1).any()
