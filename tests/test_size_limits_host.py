"""Sizes past what the kernels count in 32 bits are refused before any launch
(CPU)."""
import pytest

import paged_kv_cache_69_gb300 as pa
from paged_kv_cache_69_gb300 import build_lib as pabuild

from test_evict_host import EV
from test_int4_host import W4


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


# 2^31 bytes of codes and parameters, and where the offset of a row passes 2^32
BIG = [dict(bs=1 << 24, Hkv=2, D=128, NB=1), dict(bs=1 << 23, Hkv=8, D=128, NB=1), dict(bs=1 << 26, Hkv=1, D=64, NB=2),
       dict(bs=1 << 26, Hkv=40, D=64, NB=1)]


@pytest.mark.parametrize("over", BIG)
def test_4bit_writes_and_reads_refuse_blocks_past_32_bits(lib, over):
    a = {**W4, **over}
    sizes = [a[x] for x in ("slots", "T", "Hkv", "D", "bs", "NB")]
    assert lib.pa_reshape_and_cache(a["k"], a["v"], a["kvd"], a["key"], a["val"], a["src"], *sizes, 1.0, 1.0, None, None) == 2
    assert "2 GB" in lib.pa_last_error_detail().decode()
    assert lib.pa_gather_cache(a["key"], a["val"], a["src"], a["k"], a["v"], a["kvd"], *sizes, 1.0, 1.0, None, None) == 2
    assert "2 GB" in lib.pa_last_error_detail().decode()


@pytest.mark.parametrize("over", [dict(Hkv=1 << 20, D=128), dict(Hkv=1 << 25, D=8), dict(D=(1 << 30) + 16, kvd=pa.PA_F32)])
def test_evict_refuses_blocks_past_32_bits(lib, over):
    assert lib.pa_evict(*{**EV, "wsb": 1 << 62, **over}.values()) == 2
    assert "2 GB" in lib.pa_last_error_detail().decode()
