"""Sizes past what the kernels count in 32 bits are refused before any launch
(CPU)."""
import pytest

import paged_kv_cache_69_gb300 as pa
from paged_kv_cache_69_gb300 import build_lib as pabuild

from test_evict_host import EV


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.lib()


@pytest.mark.parametrize("budget", [(1 << 30) + 1, 2 ** 31 - 4096, 2 ** 31 - 1])
@pytest.mark.parametrize("out_of_place", [False, True])
def test_evict_refuses_a_budget_whose_positions_would_wrap(lib, budget, out_of_place):
    """A "no limit" of 2^31 - 1: the kernel's strided loops over [0, budget) would pass 2^31."""
    over = dict(budget=budget, wsb=1 << 62, **(dict(nt=256, nMB=4) if out_of_place else {}))
    assert lib.pa_evict(*{**EV, **over}.values()) == 2
    assert "budget" in lib.pa_last_error_detail().decode()
    assert lib.pa_evict_workspace_size(2, 2, 100, budget) == 0
