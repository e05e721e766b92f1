"""Tensors on 16-byte boundaries that are not 32-byte ones -- views that start 8
elements into a buffer -- in every place that the prompt, rotation and shared-prefix
calls read or write: the same bits as with tensors of their own."""
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _prompt as ref

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def shifted(t):
    """A copy of t at an address of 16 modulo 32, all else around it 7."""
    if t.numel() == 0:
        return t
    step = 16 // t.element_size()
    buf = torch.full((t.numel() + 2 * step,), 7, dtype=t.dtype, device=t.device)
    view = buf[step:step + t.numel()].view(t.shape)
    assert view.data_ptr() % 32 == 16 and view.is_contiguous()
    view.copy_(t)
    return view


def around(view):
    """What lies in front of and behind a shifted view."""
    step = 16 // view.element_size()
    flat = view._base.view(-1)
    return torch.cat([flat[:step], flat[-step:]])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(7, 1), (8, 2)])
def test_prompts(dtype, D, Hq, Hkv):
    """Rows of items that are not cut, of tokens without keys, and of cut items."""
    g = torch.Generator().manual_seed(D + Hq)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for n, lens in (([300, 1, 0, 129, 10], [300, 1, 0, 129, 4]), ([40, 3], [5000, 3]), ([9, 2], [0, 0])):
        qs, ks = ref.starts(n), ref.starts(lens)
        q, k, v = rnd(qs[-1], Hq, D), rnd(ks[-1], Hkv, D), rnd(ks[-1], Hkv, D)
        want, tol = ref.prompts(q, k, v, qs, ks, 0.2, 7.0)
        own, out = torch.full_like(q, 7), shifted(torch.full_like(q, 7))
        pa.pa_prefill(own, q, k, v, dev(qs), 0.2, k_start=dev(ks))
        pa.pa_prefill(out, shifted(q), shifted(k), shifted(v), dev(qs), 0.2, k_start=dev(ks))
        ref.check(out, want, tol)
        assert torch.equal(out, own) and (around(out) == 7).all()
        kc, vc, bt, sl = ref.paged(k, v, ks, 16, g)
        out.fill_(7)
        pa.pa_prefill_cached(out, shifted(q), shifted(kc), shifted(vc), bt, sl, dev(qs), 0.2)
        ref.check(out, want, tol)
        assert (around(out) == 7).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_shared_prefixes(dtype, D):
    g = torch.Generator().manual_seed(D)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v, q = rnd(70, 16, 2, D), rnd(70, 16, 2, D), rnd(4, 8, D)
    bt = dev([list(range(64)) + [64 + i] for i in range(4)])
    args = (bt, dev([1030, 1024, 1040, 1025]), dev([0, 4]), dev([1024]), 0.2)
    own, out = torch.empty_like(q), shifted(torch.full_like(q, 7))
    pa.pa_decode_shared(own, q, k, v, *args)
    pa.pa_decode_shared(out, shifted(q), shifted(k), shifted(v), *args)
    assert torch.equal(out, own) and (around(out) == 7).all()
    for i, L in enumerate(args[1].tolist()):
        rows = lambda x: x[bt[i].long()].view(-1, 2, D)[:L]  # noqa: E731
        ref.check(out[i:i + 1], *ref.attend(q[i:i + 1], rows(k), rows(v), 0.2, dev([L - 1])))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("kv", [None, "fp8_e4m3", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [5, 3000])                   # one row to a lane, four
def test_rotation(dtype, kv, D, T):
    g = torch.Generator().manual_seed(T + D)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    q, k, v, table = rnd(T, 8, D), rnd(T, 2, D), rnd(T, 2, D), pa.rope_table(T, D)
    pos, slots = torch.arange(T, device="cuda"), torch.randperm(T + 16, generator=g)[:T].cuda()
    NB = -(-(T + 16) // 16)
    width, of = (D // 2 + 4, torch.uint8) if kv == "int4" else (D, torch.uint8 if kv else dtype)

    def run(move):
        kc, vc = (move(torch.zeros(NB, 16, 2, width, dtype=of, device="cuda")) for _ in range(2))
        qo, ko = move(torch.zeros_like(q)), move(torch.zeros_like(k))
        pa.pa_rope_and_cache(kc, vc, qo, move(q), move(k), move(v), pos, move(table), slots, kv, key_out=ko)
        return kc, vc, qo, ko

    for a, b in zip(run(lambda t: t), run(shifted)):
        assert a.any() and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
        assert (around(b) == 7).all()
