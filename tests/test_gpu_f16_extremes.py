"""Values of the largest f16 under the prompt and shared-prefix calls: weights enter the
products rounded and the sum of weights as they are, so that a quotient may pass the
largest value by 2^-11 of it.  Outputs of finite values stay finite; infinite values that a
row attends still reach it."""
import math

import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _prompt as ref

pytestmark = pytest.mark.gpu
F16 = torch.float16
TOP = 65504.0


def dev(x, t=torch.int32):
    return torch.tensor(x, dtype=t, device="cuda")


def rows(n, Hq, D):
    """Queries for which keys of -1 in their first element lie 0.85 to 1 (log2, scale 1) below
    keys of zeros: weights that round up and ones that round down."""
    q = torch.zeros(n, Hq, D, device="cuda")
    q[..., 0] = torch.linspace(0.85 * math.log(2), math.log(2), n * Hq, device="cuda").view(n, Hq)
    return q.to(F16)


def keys(L, Hkv, D):
    k, v = torch.zeros(L, Hkv, D, dtype=F16, device="cuda"), torch.full((L, Hkv, D), TOP, dtype=F16, device="cuda")
    k[..., 0] = -1
    k[::64, :, 0] = 0                          # in every range that an item may be cut into
    v[..., 1::2] = -TOP
    return k, v


def check(out):
    """Weighted means of equal values, in f16: no more than half a step of each weight away,
    and of the output's rounding."""
    tol = (2 * 2.0 ** -11 + 2.0 ** -18) * TOP
    assert torch.isfinite(out).all()
    assert (out[..., 0::2].double() - TOP).abs().max() <= tol and (out[..., 1::2].double() + TOP).abs().max() <= tol


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,L", [(200, 1001), (700, 700), (3, 20000), (40, 9000)])      # whole items, and cut ones
def test_prompts(D, n, L):
    q, (k, v) = rows(n, 4, D), keys(L, 2, D)
    kc, vc, bt, sl = ref.paged(k, v, [0, L], 16, torch.Generator().manual_seed(n))
    for x in (None, math.inf, -math.inf):
        if x is not None:
            v[L - n, 0, 2] = vc[bt[0, (L - n) // 16], (L - n) % 16, 0, 2] = x          # every row attends it
        out, out2 = torch.empty_like(q), torch.empty_like(q)
        pa.pa_prefill(out, q, k, v, dev([0, n]), 1.0, k_start=dev([0, L]))
        pa.pa_prefill_cached(out2, q, kc, vc, bt, sl, dev([0, n]), 1.0)
        for o in (out, out2):
            if x is not None:
                assert (o[:, :2, 2] == x).all()
                o[:, :2, 2] = TOP
            check(o)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("members,shared,own", [(40, 1024, 0), (40, 1024, 300), (3, 9008, 5), (200, 304, 20)])
def test_shared_prefixes(D, members, shared, own):
    """Prefix alone, prefix and tail."""
    L, bs = shared + own, 16
    q, (k, v) = rows(members, 4, D), keys(L, 2, D)
    common, tail = shared // bs, -(-own // bs)
    kc, vc = (torch.full((common + members * tail, bs, 2, D), math.nan, dtype=F16, device="cuda") for _ in range(2))
    tables = torch.tensor([list(range(common)) + [common + i * tail + j for j in range(tail)] for i in range(members)])
    pos = torch.arange(L)
    for i in range(members):
        at = (tables[i][pos // bs].cuda(), (pos % bs).cuda())
        kc[at], vc[at] = k, v
    args = (tables.int().cuda(), dev([L] * members), dev([0, members]), dev([shared]), 1.0)
    for x in (None, math.inf, -math.inf):
        if x is not None:
            vc[0, 5, 0, 2] = x
        out = torch.empty_like(q)
        pa.pa_decode_shared(out, q, kc, vc, *args)
        if x is not None:
            assert (out[:, :2, 2] == x).all()
            out[:, :2, 2] = TOP
        check(out)


@pytest.mark.parametrize("n,L", [(200, 1001), (3, 20000)])
def test_rows_behind_the_diagonal_with_infinities(n, L):
    """An infinite value that only the last row attends: that row has it, the others the largest value."""
    q, (k, v) = rows(n, 2, 64), keys(L, 1, 64)
    v[L - 1, 0, 4] = math.inf
    out = torch.empty_like(q)
    pa.pa_prefill(out, q, k, v, dev([0, n]), 1.0, k_start=dev([0, L]))
    assert (out[-1, :, 4] == math.inf).all()
    out[-1, :, 4] = TOP
    check(out)
