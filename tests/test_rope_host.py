"""Refusals of pa_rope_and_cache: host checks (CPU)."""
import ctypes

import pytest
import torch

import paged_kv_cache_69_gb300 as pa
from paged_kv_cache_69_gb300 import build_lib as pabuild


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.lib()


def call(lib, **over):
    a = dict(kc=16, vc=16, kvd=pa.PA_F16, qo=16, ko=None, q=16, key=16, value=16, sd=pa.PA_F16, pos=16, axes=1, sec=None,
             table=16, maxp=100, rot=64, inter=0, slots=16, T=5, Hq=4, Hkv=2, D=64, bs=16, NB=8, ks=1.0, vs=1.0, err=None,
             stream=None)
    a.update(over)
    if isinstance(a["sec"], list):
        a["sec"] = (ctypes.c_int * len(a["sec"]))(*a["sec"])
    return lib.pa_rope_and_cache(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(Hq=-1), 1), (dict(maxp=0), 1), (dict(D=96), 2), (dict(rot=0), 1),
    (dict(rot=24), 1), (dict(rot=80), 1), (dict(axes=0), 2), (dict(axes=5), 2), (dict(axes=2), 1),
    (dict(axes=2, sec=[16, 15]), 1), (dict(axes=3, sec=[40, -16, 8]), 1), (dict(axes=2, sec=[2 ** 31 - 1, 2 ** 31 - 1]), 1),
    (dict(q=None), 1), (dict(qo=None), 1), (dict(key=None), 1), (dict(pos=None), 1), (dict(table=None), 1),
    (dict(slots=None), 1), (dict(kc=8), 1), (dict(ko=8), 1), (dict(table=4), 1), (dict(kvd=9), 1), (dict(kvd=pa.PA_BF16), 2),
    (dict(sd=pa.PA_FP8_E4M3, kvd=pa.PA_FP8_E4M3), 2), (dict(sd=pa.PA_INT4), 1), (dict(kvd=pa.PA_FP8_E4M3, ks=0.0), 1),
    (dict(kvd=pa.PA_FP8_E5M2, vs=float("nan")), 1), (dict(kvd=pa.PA_INT4, bs=12), 2), (dict(T=1 << 30), 2), (dict(NB=1 << 28), 2),
    (dict(kvd=pa.PA_INT4, bs=1 << 20, Hkv=64, NB=1), 2)])
def test_refusals(lib, over, status):
    assert call(lib, **over) == status
    assert lib.pa_last_error_detail().decode().startswith("rope_and_cache: ")


def test_nothing_to_do(lib):
    assert call(lib, T=0) == 0
    assert call(lib, T=0, axes=3, sec=[10, 11, 11]) == 0


def test_host_tensors_are_refused():
    z = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_rope_and_cache(torch.zeros(2, 16, 2, 64), torch.zeros(2, 16, 2, 64), z, z, z, z, torch.zeros(4, dtype=torch.int64),
                             torch.zeros(9, 64), torch.zeros(4, dtype=torch.int64))
