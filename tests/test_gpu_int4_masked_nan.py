"""Attention over 4-bit pools: a value row that holds NaN spoils the query
tokens that attend it and leaves the earlier ones, which the causal limit keeps
from it, as they are."""
import numpy as np
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _int4
from test_gpu_int4_attention import Case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa.build()


@pytest.mark.parametrize("which", ["value", "key", "both"])
@pytest.mark.parametrize("lens,counts,Hq,Hkv,D,bs,dtype", [
    ([300, 17, 64], [3, 4, 2], 4, 2, 64, 16, "f16"),
    ([129, 40], [4, 2], 28, 4, 128, 16, "bf16"),
    ([2000, 33], [16, 5], 8, 1, 128, 32, "f16"),
])
def test_a_row_of_nan_behind_the_causal_limit(lens, counts, Hq, Hkv, D, bs, dtype, which):
    c = Case(lens, Hq, Hkv, D, bs, dtype, seed=50, counts=counts)
    want, tol = c.want()
    # the newest token but one of the first sequence, KV head 0
    t = lens[0] - 2
    for k in range(2):
        if which in ("both", ("key", "value")[k]):
            code, step, low = (x.copy() for x in _int4.rows(c.pools[k]))
            step[c.tables[0][t // bs], t % bs, 0] = low[c.tables[0][t // bs], t % bs, 0] = np.float16("nan")
            c.pools[k] = _int4.pack(code, step, low)
    got = c.on_gpu().run()
    G = Hq // Hkv
    assert torch.isnan(got[counts[0] - 2:counts[0], :G]).all()
    got[counts[0] - 2:counts[0], :G] = torch.from_numpy(want[counts[0] - 2:counts[0], :G]).to(got)
    check(got, want, tol)


def test_weights_beside_a_value_row_of_nan():
    """The weights come from keys and queries alone."""
    c = Case([300], 8, 2, 128, 16, "f16", seed=51)
    w = [torch.zeros(c.NB, 2, 16, device="cuda") for _ in range(2)]
    for k in range(2):
        if k:
            code, step, low = (x.copy() for x in _int4.rows(c.pools[1]))
            step[c.tables[0][3], 2, 1] = low[c.tables[0][3], 2, 1] = np.float16("nan")
            c.pools[1] = _int4.pack(code, step, low)
        c.on_gpu()
        out = torch.empty_like(c.qd)
        pa.pa_decode_weights(out, w[k], c.qd, c.k, c.v, c.bt, c.sl, c.scale, "int4")
        torch.cuda.synchronize()
        assert torch.isnan(out[0, 4:]).all() == bool(k) and torch.isfinite(out[0, :4]).all()
    # a reference that moves elsewhere: 2^-18 for exp2, the sum and the division
    assert (w[0] - w[1]).abs().max() <= 2.0 ** -17 * w[0].max() and torch.isfinite(w[1]).all()
