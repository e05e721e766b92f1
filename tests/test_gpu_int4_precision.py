"""Attention over 4-bit pools where the steps of the value rows lie far apart:
a row with a large step and hardly any weight costs the others no bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _int4

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
D, BS = 128, 32
MANY = 912                     # sequences: more than CTAs, so that most are one segment


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa.build()


def _pools(n, q, special, seed=1):
    """K and V of n tokens (one KV head) in consecutive blocks.  special: token
    -> (score of its key, None for a random one; factor of its value's step)."""
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((n, D))
    # values with a mean per channel: what many small weights lose does not average out
    x = [0.3 * rng.standard_normal((n, D)) + rng.standard_normal(D), np.ones(n)]
    for t, (score, factor) in special.items():
        if score is not None:
            k[t] = q * score * np.sqrt(D) / (q @ q)
        x[1][t] = factor
    out = []
    for rows, f in ((k, np.ones(n)), x):
        code, step, low = _int4.encode(rows.astype(np.float32))
        step, low = ((a.astype(np.float64) * f).astype(np.float16) for a in (step, low))
        out.append(_int4.pack(*(a.reshape((n // BS, BS, 1) + a.shape[1:]) for a in (code, step, low))))
    return out


def _queries(dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(D, generator=g).to(DT[dtype])


def _decode(pools, q, n, heads, B):
    """[B, heads, D] for B sequences that share one table and hold one query in every head."""
    k, v = (torch.from_numpy(p).cuda() for p in pools)
    bt = torch.arange(n // BS, dtype=torch.int32, device="cuda").repeat(B, 1)
    sl = torch.full((B,), n, dtype=torch.int32, device="cuda")
    qd = q.cuda().repeat(B, heads, 1)
    out = torch.empty_like(qd)
    pa.pa_decode(out, qd, k, v, bt, sl, 1 / np.sqrt(D), "int4")
    torch.cuda.synchronize()
    return out


def _check(out, want, tol):
    off = np.abs(out.double().cpu().numpy() - want) - tol
    assert (off <= 0).all(), f"{(off > 0).sum()} of {off.size} beyond the bound, worst {off.max():.3g}"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [7, 16])                     # 8 and 16 query rows per warp
@pytest.mark.parametrize("n,factor", [(4096, 1000), (4096, 8000), (32768, 1000), (32768, 8000)])
@pytest.mark.parametrize("where", ["first", "inside", "last"])
def test_a_large_step_without_weight(dtype, heads, n, factor, where):
    """One key takes half of the softmax, the row with the large step e^-60 of
    it.  (Both are multiples of 128 tokens in: one warp's, of the four that share
    a chunk.)"""
    q = _queries(dtype)
    t = {"first": 0, "inside": n // 2, "last": n - 128}[where]
    pools = _pools(n, q.double().numpy(), {128: (np.log(n) + 0.5, 1), t: (-60.0, factor)})
    table = np.arange(n // BS)[None]
    want, tol = _int4.attention(q.double().numpy().reshape(1, 1, D), pools, table, [n], 1 / np.sqrt(D), None, dtype)
    _check(_decode(pools, q, n, heads, MANY), want, tol)


@pytest.mark.parametrize("counts", [4, 5])
def test_a_large_step_that_only_the_last_query_may_see(counts):
    """Causal masking hides the last token's value from the queries before it."""
    n, B = 4096, 400
    q = _queries("f16")
    pools = _pools(n, q.double().numpy(), {31: (np.log(n) + 0.5, 1), n - 1: (None, 8000)})
    table = np.arange(n // BS)[None]
    qs = q.repeat(counts, 1, 1)
    want, tol = _int4.attention(qs.double().numpy(), pools, table, [n], 1 / np.sqrt(D), [0, counts], "f16")
    k, v = (torch.from_numpy(p).cuda() for p in pools)
    bt = torch.arange(n // BS, dtype=torch.int32, device="cuda").repeat(B, 1)
    sl = torch.full((B,), n, dtype=torch.int32, device="cuda")
    start = torch.arange(0, B * counts + 1, counts, dtype=torch.int32, device="cuda")
    for heads in (2, 7):
        qd = qs.repeat(B, heads, 1).cuda()
        out = torch.empty_like(qd)
        pa.pa_attention(out, qd, k, v, bt, sl, start, 1 / np.sqrt(D), counts, "int4")
        torch.cuda.synchronize()
        _check(out.view(B, counts, heads, D), want[None], tol[None])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("score", [20.0, 80.0])
def test_a_value_of_zeros_that_takes_nearly_all_weight(dtype, score):
    """Its step is 0; the others' products are all there is of the output (nothing at 80: e^-80 of each)."""
    n = 4096
    q = _queries(dtype)
    pools = _pools(n, q.double().numpy(), {0: (score, 0)})
    table = np.arange(n // BS)[None]
    want, tol = _int4.attention(q.double().numpy().reshape(1, 1, D), pools, table, [n], 1 / np.sqrt(D), None, dtype)
    for B in (1, MANY):
        _check(_decode(pools, q, n, 7, B), want, tol)


@pytest.mark.parametrize("factor", [2.0 ** -12, 8000])
def test_weights_beside_steps_that_lie_apart(factor):
    """pa_decode_weights: the softmax weights do not depend on the values' steps."""
    n, G = 32768, 7
    q = _queries("f16")
    half = n // 2
    pools = _pools(n, q.double().numpy(), {half: (np.log(n) + 0.5, factor), 5: (-60.0, 8000), n - 1: (3.0, 0)})
    table = np.arange(n // BS)[None]
    q64, scale = q.double().numpy(), 1 / np.sqrt(D)
    want, tol = _int4.attention(q64.reshape(1, 1, D), pools, table, [n], scale, None, "f16")
    kv, ka = (a.reshape(n, D) for a in _int4.values(pools[0]))
    s = kv @ q64 * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    # scores: D products in f32; a weight moves by twice that, and 2^-18 for exp2, the sums and the division;
    # G of them are added in f32
    rel = 2 * (D + 2) * 2.0 ** -23 * (ka @ np.abs(q64)).max() * scale + 2.0 ** -18 + (G + 1) * 2.0 ** -24
    k, v = (torch.from_numpy(x).cuda() for x in pools)
    w = torch.zeros(n // BS, 1, BS, device="cuda")
    qd = q.cuda().repeat(1, G, 1)
    out = torch.empty_like(qd)
    pa.pa_decode_weights(out, w, qd, k, v, torch.from_numpy(table.astype(np.int32)).cuda(),
                         torch.tensor([n], dtype=torch.int32, device="cuda"), scale, "int4")
    torch.cuda.synchronize()
    _check(out, want, tol)
    _check(w.view(-1), G * p, rel * G * p + 2.0 ** -120)
