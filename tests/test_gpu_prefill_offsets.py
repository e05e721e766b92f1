"""Sequences of pa_prefill and pa_prefill_cached whose entries do not fit: their rows are left
as they are, those of the others are right."""
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _prompt as ref
from test_gpu_prefill import F16, Case

pytestmark = pytest.mark.gpu


def _check(c, out, skipped):
    want, tol = ref.prompts(c.q, c.k, c.v, c.qs, c.ks, c.scale, 7.0)
    assert c.err.item() == pa.ERRBIT_BAD_QUERY
    a, b = c.qs[skipped], c.qs[skipped + 1]
    assert (out[a:b] == 7).all()
    want[a:b], tol[a:b] = 7.0, 0.0
    ref.check(out, want, tol)


@pytest.mark.parametrize("bad,skipped", [([0, 30, 230, 331], 2), ([0, 30, 230, 2 ** 31 - 1], 2), ([-1, 30, 230, 330], 0),
                                         ([-2 ** 31, 30, 230, 330], 0), ([31, 30, 230, 330], 0), ([0, 30, 230, 229], 2)])
def test_query_rows(bad, skipped):
    c = Case([300, 200, 100], 4, 2, 64, F16, q_lens=[30, 200, 100])
    kc, vc, bt, lens = c.pools(16)
    for call in (lambda o: pa.pa_prefill(o, c.q, c.k, c.v, c.dev(bad), c.scale, k_start=c.k_start, err_flag=c.err),
                 lambda o: pa.pa_prefill_cached(o, c.q, kc, vc, bt, lens, c.dev(bad), c.scale, err_flag=c.err)):
        c.err.zero_()
        out = torch.full_like(c.q, 7.0)
        call(out)
        _check(c, out, skipped)


@pytest.mark.parametrize("bad,skipped", [([0, 300, 500, 601], 2), ([0, 300, 500, 2 ** 31 - 1], 2), ([-1, 300, 500, 600], 0),
                                         ([0, 300, 500, 499], 2), ([301, 300, 500, 600], 0)])
def test_key_rows(bad, skipped):
    c = Case([300, 200, 100], 4, 2, 64, F16, q_lens=[30, 200, 100])
    out = torch.full_like(c.q, 7.0)
    pa.pa_prefill(out, c.q, c.k, c.v, c.dev(c.qs), c.scale, k_start=c.dev(bad), err_flag=c.err)
    _check(c, out, skipped)


def test_key_rows_that_only_the_query_offsets_say():
    """No k_start: sequences whose query rows lie behind the last key row."""
    c = Case([30, 200, 100], 4, 2, 64, F16)
    out = torch.full_like(c.q, 7.0)
    pa.pa_prefill(out, c.q, c.k[:329].contiguous(), c.v[:329].contiguous(), c.dev(c.qs), c.scale, err_flag=c.err)
    _check(c, out, 2)
