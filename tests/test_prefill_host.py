"""Refusals of pa_prefill and pa_prefill_cached: host checks (CPU)."""
import pytest
import torch

import paged_kv_cache_69_gb300 as pa
from paged_kv_cache_69_gb300 import build_lib as pabuild


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.lib()


def flat(lib, **over):
    a = dict(out=16, q=16, k=16, v=16, dt=pa.PA_F16, qs=16, ks=None, B=2, T=10, Tk=10, Hq=4, Hkv=2, D=128, scale=0.1, ws=256,
             wsb=1 << 40, err=None, stream=None)
    a.update(over)
    return lib.pa_prefill(*a.values())


def cached(lib, **over):
    a = dict(out=16, q=16, qd=pa.PA_F16, k=16, v=16, kvd=pa.PA_F16, bt=16, mb=4, sl=16, qs=16, B=2, T=10, Hq=4, Hkv=2, D=128,
             bs=16, NB=8, scale=0.1, ws=256, wsb=1 << 40, err=None, stream=None)
    a.update(over)
    return lib.pa_prefill_cached(*a.values())


COMMON = [(dict(Hq=5), 1), (dict(D=96), 2), (dict(D=0), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(v=8), 1),
          (dict(qs=None), 1), (dict(B=-1), 1), (dict(T=-1), 1), (dict(Hq=258, Hkv=2), 2), (dict(Hq=512, Hkv=512), 2),
          (dict(T=1 << 30), 2)]


@pytest.mark.parametrize("over,status", COMMON + [(dict(dt=pa.PA_F32), 2), (dict(dt=pa.PA_FP8_E4M3), 2), (dict(dt=17), 1),
                                                  (dict(Tk=-1), 1), (dict(Tk=1 << 30), 2)])
def test_refusals(lib, over, status):
    assert flat(lib, **over) == status
    assert lib.pa_last_error_detail().decode().startswith("prefill: ")


@pytest.mark.parametrize("over,status", COMMON + [(dict(kvd=pa.PA_BF16), 2), (dict(kvd=pa.PA_INT4), 2), (dict(bs=48), 2),
                                                  (dict(bt=None), 1), (dict(sl=None), 1), (dict(mb=0), 1), (dict(NB=0), 1),
                                                  (dict(NB=1 << 27), 2), (dict(mb=1 << 26), 2)])
def test_refusals_cached(lib, over, status):
    assert cached(lib, **over) == status
    assert lib.pa_last_error_detail().decode().startswith("prefill_cached: ")


def test_nothing_to_do(lib):
    assert flat(lib, B=0) == 0 and flat(lib, T=0) == 0
    assert cached(lib, B=0) == 0 and cached(lib, T=0) == 0


def test_workspace_size_of_bad_sizes(lib):
    for a in ((-1, 5, 4, 2, 64), (2, -5, 4, 2, 64), (2, 5, 0, 2, 64), (2, 5, 5, 2, 64), (2, 5, 4, 0, 64), (2, 5, 4, 2, 0),
              (2, 5, 129, 1, 64)):
        assert lib.pa_prefill_workspace_size(*a) == 0


def test_host_tensors_are_refused():
    q, k = torch.zeros(4, 4, 64), torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_prefill(q, q, k, k, torch.zeros(2, dtype=torch.int32), 1.0)
