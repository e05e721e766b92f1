"""4-bit pools whose byte offsets pass 32 bits: every call on blocks at the end
of such a pool gives what it gives on a small copy of them."""
import torch
import pytest

import paged_kv_cache_69_gb300 as pa

pytestmark = pytest.mark.gpu


def test_pools_of_more_than_four_gigabytes():
    pa.build()
    NB, bs, Hkv, D, n = 640000, 16, 8, 128, 20         # 5.6 GB per pool
    k = pa.alloc_int4_cache(NB, bs, Hkv, D)
    v = torch.zeros_like(k)
    last = torch.arange(NB - 1, NB - 1 - n, -1, device="cuda")
    L = n * bs - 5
    pos = torch.arange(L, device="cuda")
    x, y = torch.randn(L, Hkv, D, device="cuda").half(), torch.randn(L, Hkv, D, device="cuda").half()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_reshape_and_cache(k, v, x, y, last[pos // bs] * bs + pos % bs, "int4", err_flag=err)
    sides = [(k, v, torch.zeros(NB, Hkv, bs, device="cuda"), last)]
    sides.append((k[last], v[last], torch.zeros(n, Hkv, bs, device="cuda"), torch.arange(n, device="cuda")))
    q = torch.randn(1, 32, D, device="cuda").half()
    sl = torch.tensor([L], dtype=torch.int32, device="cuda")
    got = []
    for kc, vc, w, blocks in sides:
        a, b, o, o2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(q), torch.empty_like(q)
        bt, nl = blocks.int().view(1, -1), torch.empty_like(sl)
        pa.pa_gather_cache(a, b, kc, vc, blocks[pos // bs] * bs + pos % bs, "int4", err_flag=err)
        pa.pa_decode(o, q, kc, vc, bt, sl, 0.09, "int4", err_flag=err)
        pa.pa_decode_weights(o2, w, q, kc, vc, bt, sl, 0.09, "int4", err_flag=err)
        added = w[blocks].clone()
        pa.pa_evict(kc, vc, w, bt, sl, nl, 100, "int4", num_sink=2, num_recent=20, err_flag=err)
        got.append((a, b, o, o2, added, kc[blocks], vc[blocks], w[blocks], nl))
    for p, r in zip(*got):
        assert torch.equal(p, r)
    # half a step of a row of 128 normal values, and their rounding
    assert (got[0][0] - x).abs().max() < 0.4 and err.item() == 0 and got[0][2].any()
