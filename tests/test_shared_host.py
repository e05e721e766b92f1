"""Refusals of pa_decode_shared: host checks (CPU)."""
import pytest
import torch

import paged_kv_cache_69_gb300 as pa
from paged_kv_cache_69_gb300 import build_lib as pabuild


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.lib()


def call(lib, **over):
    a = dict(out=16, q=16, qd=pa.PA_F16, k=16, v=16, kvd=pa.PA_F16, bt=16, mb=4, sl=16, gs=16, pl=16, B=4, NG=2, Hq=4, Hkv=2,
             D=128, bs=16, NB=8, scale=0.1, ws=256, wsb=1 << 40, err=None, stream=None)
    a.update(over)
    return lib.pa_decode_shared(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), 1), (dict(NG=-1), 1), (dict(Hq=5), 1), (dict(Hkv=0), 1), (dict(mb=0), 1), (dict(NB=0), 1), (dict(D=96), 2),
    (dict(bs=48), 2), (dict(q=None), 1), (dict(gs=None), 1), (dict(pl=None), 1), (dict(sl=None), 1), (dict(bt=None), 1),
    (dict(out=8), 1), (dict(kvd=pa.PA_BF16), 2), (dict(qd=pa.PA_F32, kvd=pa.PA_F32), 2), (dict(kvd=pa.PA_FP8_E4M3), 2),
    (dict(kvd=pa.PA_INT4), 2), (dict(qd=12), 1), (dict(Hq=258), 2), (dict(Hq=512, Hkv=512), 2), (dict(NB=1 << 27), 2),
    (dict(mb=1 << 26), 2), (dict(B=1 << 30), 2)])
def test_refusals(lib, over, status):
    assert call(lib, **over) == status
    assert lib.pa_last_error_detail().decode().startswith("decode_shared: ")


def test_nothing_to_do(lib):
    assert call(lib, B=0) == 0 and call(lib, B=0, NG=0) == 0


def test_workspace_size_of_bad_sizes(lib):
    for a in ((-1, 1, 4, 2, 100, 64), (2, -1, 4, 2, 100, 64), (2, 1, 0, 2, 100, 64), (2, 1, 5, 2, 100, 64),
              (2, 1, 4, 0, 100, 64), (2, 1, 4, 2, -1, 64), (2, 1, 4, 2, 100, 0), (2, 1, 129, 1, 100, 64)):
        assert lib.pa_decode_shared_workspace_size(*a) == 0


def test_host_tensors_are_refused():
    z, i = torch.zeros(4, 2, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_decode_shared(z, z, torch.zeros(2, 16, 2, 64), torch.zeros(2, 16, 2, 64), i.view(1, 2), i, i, i[:1], 1.0)
