"""pa_decode_weights where a head's scores are all -infinity: the output is 0,
as pa_decode's, and nothing is added."""
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa.build()


@pytest.mark.parametrize("kv", ["f32", "f16", "bf16", "fp8_e5m2"])
@pytest.mark.parametrize("n", [3, 5000])                # one segment, and a merge
def test_a_head_without_scores_adds_nothing(kv, n):
    D, NB = 128, -(-n // 16)
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "fp8_e5m2": torch.float8_e5m2}[kv]
    qd = torch.float16 if kv == "fp8_e5m2" else dt
    k = torch.zeros(NB, 16, 2, D, device="cuda")
    k[:, :, 0, 5] = -float("inf")
    k, v = k.to(dt), torch.ones(NB, 16, 2, D, device="cuda").to(dt)
    q = torch.ones(1, 8, D, dtype=qd, device="cuda")
    bt = torch.arange(NB, dtype=torch.int32, device="cuda").view(1, -1)
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, ref = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    w = torch.full((NB, 2, 16), 3.0, device="cuda")
    pa.pa_decode(ref, q, k, v, bt, sl, 0.1)
    for _ in range(2):                                   # the second call adds to the first's
        pa.pa_decode_weights(out, w, q, k, v, bt, sl, 0.1)
    # (pa_decode's own fp8 kernel carries a query as two terms, and 0 times an infinite key is none)
    assert not out[0, :4].any() and (kv == "fp8_e5m2" or not ref[0, :4].any())
    flat = w.transpose(0, 1).reshape(2, -1)
    assert (flat[0, :n - 1] == 3.0).all() and flat[0, n - 1] == 0.0 and (flat[:, n:] == 3.0).all()
    # four heads of equal weights each; the newest token's entry starts from 0 in both calls
    want = torch.full((n,), 3.0 + 2 * 4 / n, device="cuda")
    want[-1] = 4 / n
    assert (flat[1, :n] - want).abs().max() <= 2.0 ** -18 * want.max()
