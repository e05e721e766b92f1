"""pa_evict and pa_decode_weights on the host: the reference selection on
worked cases, the binding's marshalling and refusals, the library's argument
checks (CPU)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_69_gb300 as pa
from paged_kv_cache_69_gb300 import build_lib as pabuild

import _evict
from test_abi_host import _decode_args
from test_binding_host import _decode_inputs, _pool, rec  # noqa: F401


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.lib()


def test_reference_on_worked_cases():
    w = [5, 1, 4, 2, 3, 0, 9, 7]
    # budget 5, one sink, two recent: 0 | 2 and 4 of 1..5 | 6 7; place 1 takes 4 (the kept row from behind 3)
    assert _evict.kept_positions(w, 5, 1, 2) == [0, 4, 2, 6, 7]
    assert _evict.kept_positions(w, 8, 0, 0) == list(range(8))
    assert _evict.kept_positions(w, 3, 0, 0) == [0, 6, 7]
    assert _evict.kept_positions(w, 2, 0, 2) == [6, 7]
    assert _evict.kept_positions([1.0] * 6, 3, 0, 1) == [0, 1, 5]                # ties: the lower positions
    assert _evict.kept_positions([float("nan"), -1.0, 2.0], 2, 0, 0) == [2, 1]
    assert _evict.kept_positions([float("nan"), float("-inf"), 2.0], 2, 0, 0) == [2, 1]


def test_reference_keeps_distinct_rows_and_the_largest_sum():
    rng = np.random.default_rng(0)
    for _ in range(200):
        L = int(rng.integers(1, 60))
        budget = int(rng.integers(1, 60))
        recent = int(rng.integers(0, budget + 1))
        sink = int(rng.integers(0, budget - recent + 1))
        w = rng.random(L).tolist()
        got = _evict.kept_positions(w, budget, sink, recent)
        assert len(set(got)) == len(got) == min(L, budget)
        if L > budget:
            assert set(range(sink)) <= set(got) and set(range(L - recent, L)) <= set(got)
            mid = [w[t] for t in got if sink <= t < L - recent]
            assert sorted(mid) == sorted(sorted(w[sink:L - recent], reverse=True)[:budget - sink - recent])


def _evict_tensors(B=3, NB=10, bs=16, Hkv=2):
    k, v = _pool(NB, bs, Hkv)
    return dict(k_cache=k, v_cache=v, weights=torch.zeros(NB, Hkv, bs), block_tables=torch.zeros(B, 5, dtype=torch.int32),
                seq_lens=torch.full((B,), 70, dtype=torch.int32), new_seq_lens=torch.zeros(B, dtype=torch.int32), budget=48)


def test_evict_passes_the_sizes(rec):  # noqa: F811
    a = _evict_tensors()
    pa.pa_evict(**a, num_sink=2, num_recent=9)
    (n0, w), (n1, c) = rec.calls
    assert n0 == "pa_evict_workspace_size" and w == (3, 2, 80, 48)
    # kv_dtype, MB, new tables, kept, B, Hkv, D, bs, NB, budget, sink, recent, workspace bytes
    assert n1 == "pa_evict" and (c[2], c[5], c[7], c[8], c[10]) == (pa.PA_F16, 5, None, 0, None)
    assert c[11:19] == (3, 2, 64, 16, 10, 48, 2, 9) and c[20] == 4096
    new = torch.zeros(4, 3, dtype=torch.int32)
    pa.pa_evict(**a, new_block_tables=new)
    assert rec.calls[-1][1][8] == 3 and rec.calls[-1][1][7] is not None
    pa.pa_evict(**a, new_block_tables=a["block_tables"])          # the same tables: in place
    assert rec.calls[-1][1][7] is None


@pytest.mark.parametrize("over", [
    dict(weights=torch.zeros(10, 16, 2)), dict(weights=torch.zeros(10, 2, 16, dtype=torch.float16)),
    dict(new_seq_lens=torch.zeros(3)), dict(new_seq_lens=torch.zeros(2, dtype=torch.int32)),
    dict(kept=torch.zeros(3, 2, 47, dtype=torch.int32)), dict(kept=torch.zeros(3, 2, 48)),
    dict(new_block_tables=torch.zeros(2, 3, dtype=torch.int32)), dict(new_block_tables=torch.zeros(3, 3)),
    dict(block_tables=torch.zeros(2, 5, dtype=torch.int32)), dict(kv_dtype="int4"),
])
def test_evict_rejects_inconsistent_tensors(rec, over):  # noqa: F811
    with pytest.raises(ValueError):
        pa.pa_evict(**{**_evict_tensors(), **over})
    assert not rec.calls


def test_decode_weights_passes_the_sizes_and_checks(rec):  # noqa: F811
    k, v = _pool()
    q, out, bt, sl = _decode_inputs()
    w = torch.zeros(10, 2, 16)
    pa.pa_decode_weights(out, w, q, k, v, bt, sl, 0.125)
    (n0, a0), (n1, a1) = rec.calls
    assert n0 == "pa_decode_weights_workspace_size" and a0 == (3, 4, 80, 64)
    assert n1 == "pa_decode_weights" and (a1[3], a1[6], a1[8], a1[10]) == (pa.PA_F16, pa.PA_F16, 5, None)
    assert a1[11:18] == (3, 4, 2, 64, 16, 10, 0.125) and a1[21] == 4096
    n = len(rec.calls)
    for over in (dict(weights=w.double()), dict(weights=torch.zeros(10, 16, 2)),
                 dict(fresh=torch.ones(3)), dict(fresh=torch.ones(2, dtype=torch.int32)), dict(out=out.float()),
                 dict(seq_lens=sl.long()), dict(block_tables=bt[:2])):
        a = dict(out=out, weights=w, q=q, k_cache=k, v_cache=v, block_tables=bt, seq_lens=sl, scale=0.1)
        with pytest.raises(ValueError):
            pa.pa_decode_weights(**{**a, **over})
    assert len(rec.calls) == n


EV = dict(k=256, v=256, kvd=pa.PA_F16, w=256, bt=256, MB=4, sl=256, nt=None, nMB=0, nl=256, kept=None, B=2, Hkv=2, D=64,
          bs=16, NB=8, budget=32, sink=1, recent=4, ws=256, wsb=1 << 20, err=None, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(budget=0), 1), (dict(sink=-1), 1), (dict(recent=-1), 1), (dict(sink=20, recent=13), 1),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), 1),
    (dict(B=-1), 1), (dict(w=None), 1), (dict(nl=None), 1), (dict(bt=None), 1), (dict(w=260), 1), (dict(k=8), 1),
    (dict(kvd=7), 1), (dict(nt=256, nMB=0), 1), (dict(bs=24), 2), (dict(kvd=pa.PA_INT4, D=96), 2), (dict(D=4), 2),
    (dict(MB=1 << 27), 2), (dict(NB=1 << 28), 2),
    (dict(ws=None), 3), (dict(wsb=16), 3), (dict(ws=264), 3),
])
def test_evict_host_validation(lib, over, status):
    assert lib.pa_evict(*{**EV, **over}.values()) == status
    assert lib.pa_last_error_detail().decode() != ""


def test_evict_of_no_sequences_is_a_noop_and_sizes_reject_nonsense(lib):
    assert lib.pa_evict(*{**EV, "B": 0}.values()) == 0
    assert lib.pa_evict_workspace_size(2, 0, 100, 10) == 0 and lib.pa_evict_workspace_size(2, 2, 100, 0) == 0
    assert lib.pa_evict_workspace_size(2, 2, 100, 10) > 0
    assert lib.pa_decode_weights_workspace_size(-1, 4, 100, 128) == 0


@pytest.mark.parametrize("over,status", [(dict(Hq=5), 1), (dict(D=96), 2), (dict(q=None), 1), (dict(kvd=pa.PA_BF16), 2),
                                         (dict(B=-1), 1), (dict(w=None), 1), (dict(w=8), 1)])
def test_decode_weights_host_validation(lib, over, status):
    over = dict(over)
    w = over.pop("w", 256)
    a = _decode_args(**over)
    # out, weights, q ... seq_lens, fresh, sizes, scales, workspace ... (no partition_tokens)
    args = (a[0], w) + a[1:9] + (None,) + a[9:18] + a[19:]
    assert lib.pa_decode_weights(*args) == status
    assert lib.pa_last_error_detail().decode() != ""


def test_decode_weights_of_no_sequences_is_a_noop(lib):
    a = _decode_args(B=0)
    assert lib.pa_decode_weights(a[0], None, *a[1:9], None, *a[9:18], *a[19:]) == 0


def test_tensors_of_another_device_are_refused(monkeypatch):
    class OnDevice:
        is_cuda = True

        def __init__(self, index):
            self.index = index

        def is_contiguous(self):
            return True

        def get_device(self):
            return self.index

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    pa._dev(OnDevice(1), None, OnDevice(1))
    for bad in ((OnDevice(0),), (OnDevice(1), OnDevice(0))):
        with pytest.raises(ValueError):
            pa._dev(*bad)
    with pytest.raises(ValueError):
        pa._dev(torch.zeros(2))


def test_decode_weights_refuses_more_sequences_than_its_grid(lib):
    a = _decode_args(B=65536)
    assert lib.pa_decode_weights(a[0], 256, *a[1:9], None, *a[9:18], *a[19:]) == 2
