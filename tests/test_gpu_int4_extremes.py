"""Rows of a 4-bit cache that reach the largest f16 values: what is read back
and attended as f16 stays finite."""
import numpy as np
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _int4

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa.build()


def _pools(src, D, n):
    """n tokens of one head whose values alternate between the two largest, and
    infinities in the last (f32, bf16: as far as they go)."""
    x = torch.where(torch.arange(D) % 2 == 0, 65504.0, -65504.0).repeat(n, 1, 1)
    x[-1] *= float("inf") if src == "f16" else 1e30
    x = x.to(DT[src]).cuda()
    k, v = (pa.alloc_int4_cache(-(-n // 16), 16, 1, D) for _ in range(2))
    pa.pa_reshape_and_cache(k, v, torch.zeros_like(x), x, torch.arange(n, device="cuda"), "int4")
    return k, v


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dst", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_read_back(src, dst, D):
    k, v = _pools(src, D, 5)
    value = _int4.values(v.cpu().numpy())[0].reshape(16, D)[:5]
    assert value.max() == 65536 and value.min() == -65504            # the step is rounded up
    a, b = (torch.empty(5, 1, D, dtype=DT[dst], device="cuda") for _ in range(2))
    pa.pa_gather_cache(a, b, k, v, torch.arange(5, device="cuda"), "int4")
    want = torch.from_numpy(np.clip(value, -65504, 65504) if dst == "f16" else value).to(DT[dst])
    assert torch.equal(b[:, 0].cpu(), want) and not a.any()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [1, 20, 30000])                         # written directly, and by the merge
def test_attention(dtype, n):
    D = 128
    k, v = _pools("f32", D, n)
    q = torch.ones(1, 4, D, dtype=DT[dtype], device="cuda")
    bt = torch.arange(k.shape[0], dtype=torch.int32, device="cuda").view(1, -1)
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    pa.pa_decode(out, q, k, v, bt, sl, 0.1, "int4")
    w = torch.zeros(k.shape[0], 1, 16, device="cuda")
    out2 = torch.empty_like(q)
    pa.pa_decode_weights(out2, w, q, k, v, bt, sl, 0.1, "int4")
    for o in (out, out2):
        assert torch.isfinite(o).all()
        # f16 products and the output's type: half a step of each
        tol = (2.0 ** -11 + 2.0 ** -18 + _int4.UNIT_OUT[dtype]) * 65536
        assert (o[..., 0::2].float() - 65536).abs().max() <= tol and (o[..., 1::2].float() + 65504).abs().max() <= tol
    if dtype == "f16" and n == 1:
        assert (out[..., 0::2] == 65504).all()


def test_a_row_of_nan_is_still_nan():
    k, v = _pools("f16", 64, 3)
    x = torch.full((1, 1, 64), float("nan"), dtype=torch.float16, device="cuda")
    pa.pa_reshape_and_cache(k, v, x, x, torch.tensor([1], device="cuda"), "int4")
    a, b = (torch.empty(3, 1, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.pa_gather_cache(a, b, k, v, torch.arange(3, device="cuda"), "int4")
    assert torch.isnan(a[1]).all() and torch.isnan(b[1]).all() and torch.isfinite(b[[0, 2]]).all()
