"""Values of the largest f16 in f16 pools under the decode calls and pa_attention: outputs of
finite values stay finite, infinite values that a row attends still reach it."""
import math

import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _prompt as ref
from test_gpu_f16_extremes import TOP, check, dev, keys, rows

pytestmark = pytest.mark.gpu


def _calls(q, kc, vc, bt, sl, MB, parts):
    """Every call that attends with one query per sequence, by name."""
    out = {}
    for pt in (0, parts):
        o = out[f"pa_decode {pt}"] = torch.empty_like(q)
        pa.pa_decode(o, q, kc, vc, bt, sl, 1.0, partition_tokens=pt)
    o = out["pa_decode_noalloc"] = torch.empty_like(q)
    pa.pa_decode_noalloc(o, q, kc, vc, bt, sl, 1.0)
    o = out["pa_decode_weights"] = torch.empty_like(q)
    pa.pa_decode_weights(o, torch.zeros(kc.shape[0], kc.shape[2], kc.shape[1], device="cuda"), q, kc, vc, bt, sl, 1.0)
    o = out["pa_attention"] = torch.empty_like(q)
    pa.pa_attention(o, q, kc, vc, bt, sl, torch.arange(q.shape[0] + 1, dtype=torch.int32, device="cuda"), 1.0, 1)
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,L", [(400, 150), (3, 20000), (1, 9000)])               # written directly, and by the merge
def test_decode(D, B, L):
    q, (k, v) = rows(B, 8, D), keys(L, 2, D)
    kc, vc, bt, sl = ref.paged(k, v, [0, L], 16, torch.Generator().manual_seed(L))
    bt, sl = bt.repeat(B, 1).contiguous(), sl.repeat(B)
    for x in (None, math.inf, -math.inf):
        if x is not None:
            vc[bt[0, 0], 5, 0, 2] = x
        for name, out in _calls(q, kc, vc, bt, sl, bt.shape[1], 256).items():
            if x is not None:
                assert (out[:, :4, 2] == x).all(), name
                out[:, :4, 2] = TOP
            check(out)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,heads", [(8, 4), (30, 4), (16, 14)])                    # mma.sync, tcgen05
@pytest.mark.parametrize("L", [200, 20000])
def test_attention(D, n, heads, L):
    B = 6
    q, (k, v) = rows(B * n, heads, D), keys(L, 2, D)
    kc, vc, bt, sl = ref.paged(k, v, [0, L], 16, torch.Generator().manual_seed(L))
    out = torch.empty_like(q)
    pa.pa_attention(out, q, kc, vc, bt.repeat(B, 1).contiguous(), sl.repeat(B), dev(list(range(0, B * n + 1, n))), 1.0, n)
    check(out)
