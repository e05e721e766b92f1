"""The 4-bit cache on the host: the reference format against exact rational
arithmetic, the binding's marshalling and refusals, the library's argument
checks (CPU)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_69_gb300 as pa
from paged_kv_cache_69_gb300 import build_lib as pabuild

import _int4
from test_binding_host import rec  # noqa: F401  (the recording stand-in)


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.lib()


def _nearest_half(x: Fraction) -> np.float16:
    """The float16 nearest to an exact rational, ties to the even one, by search."""
    h = np.arange(0x7C00, dtype=np.uint16).view(np.float16)
    k = int(np.searchsorted(h.astype(np.float64), float(abs(x))))
    best = min((i for i in range(max(0, k - 2), min(len(h), k + 3))),
               key=lambda i: (abs(Fraction(float(h[i])) - abs(x)), i & 1))
    return np.float16(-h[best]) if x < 0 else h[best]


@pytest.mark.parametrize("seed", range(4))
def test_reference_rounds_exact_quotients(seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((6, 32)) * 10.0 ** rng.uniform(-5, 4, (6, 1))).astype(np.float32)
    x[0] = rng.integers(-8, 8, 32) / 2                       # quotients that are halves exactly
    code, step, low = _int4.encode(x)
    for r in range(x.shape[0]):
        xs = [Fraction(float(v)) for v in x[r]]
        lo = _nearest_half(min(xs))
        st = _nearest_half((max(xs) - Fraction(float(lo))) / 15)
        assert low[r] == lo and step[r] == st
        for v, c in zip(xs, code[r]):
            want = round((v - Fraction(float(lo))) / Fraction(float(st)))    # half to even
            assert c == min(max(want, 0), 15)


def test_reference_error_is_at_most_half_a_step():
    rng = np.random.default_rng(9)
    x = rng.standard_normal((50, 128)).astype(np.float16)
    code, step, low = _int4.encode(x)
    err = np.abs(_int4.decode(code, step, low) - x.astype(np.float64))
    # half a step, plus what rounding low up and step down may cut off at the ends
    s, l64 = step.astype(np.float64), np.abs(low.astype(np.float64))
    assert (err.max(-1) <= 0.5 * s + 2.0 ** -11 * l64 + 15 * 2.0 ** -11 * s).all()


def test_pool_layout_round_trip():
    rng = np.random.default_rng(1)
    code = rng.integers(0, 16, (3, 8, 2, 64)).astype(np.uint8)
    step, low = rng.standard_normal((2, 3, 8, 2)).astype(np.float16)
    pool = _int4.pack(code, step, low)
    assert pool.shape == (3, 8, 2, 36)
    c, s, lo = _int4.rows(pool)
    assert (c == code).all() and (s == step).all() and (lo == low).all()
    # dimension 2b in the low nibble of byte b, heads outside tokens, parameters behind all codes
    flat = pool.reshape(3, -1)
    assert flat[1, (1 * 8 + 5) * 32 + 7] == code[1, 5, 1, 14] | (code[1, 5, 1, 15] << 4)
    par = flat[2, 2 * 8 * 32:].copy().view(np.float16)
    assert par[2 * (1 * 8 + 3)] == step[2, 3, 1] and par[2 * (1 * 8 + 3) + 1] == low[2, 3, 1]


def _pool4(NB=10, bs=16, Hkv=2, D=64):
    return torch.zeros(NB, bs, Hkv, D // 2 + 4, dtype=torch.uint8), torch.zeros(NB, bs, Hkv, D // 2 + 4, dtype=torch.uint8)


def test_binding_sizes_of_4bit_pools(rec):  # noqa: F811
    k, v = _pool4()
    key = torch.zeros(7, 2, 64, dtype=torch.bfloat16)
    slots = torch.arange(7)
    pa.pa_reshape_and_cache(k, v, key, key.clone(), slots, "int4")
    a = rec.calls[-1][1]
    assert (a[2], a[5], a[7], a[8], a[9], a[10], a[11]) == (pa.PA_INT4, pa.PA_BF16, 7, 2, 64, 16, 10)
    pa.pa_gather_cache(key, key.clone(), k, v, slots, "int4")
    name, a = rec.calls[-1]
    assert name == "pa_gather_cache"
    assert (a[2], a[5], a[7], a[8], a[9], a[10], a[11]) == (pa.PA_BF16, pa.PA_INT4, 7, 2, 64, 16, 10)
    pairs = torch.tensor([[1, 2]])
    pa.pa_copy_blocks(k, v, pairs, "int4")
    a = rec.calls[-1][1]
    assert (a[2], a[4], a[5], a[6], a[7], a[8]) == (pa.PA_INT4, 1, 2, 64, 16, 10)
    pa.pa_copy_blocks_layers([k, k.clone()], [v, v.clone()], pairs, pa.PA_INT4)
    a = rec.calls[-1][1]
    assert (a[2], a[3], a[5], a[6], a[7], a[8], a[9]) == (2, pa.PA_INT4, 1, 2, 64, 16, 10)


def test_binding_refuses_other_pools_as_4bit(rec):  # noqa: F811
    k, v = _pool4()
    key = torch.zeros(7, 2, 64, dtype=torch.bfloat16)
    slots = torch.arange(7)
    with pytest.raises(ValueError):                      # not uint8
        pa.pa_reshape_and_cache(k.short(), v.short(), key, key, slots, "int4")
    with pytest.raises(ValueError):                      # head_dim of the rows is not the pool's
        pa.pa_reshape_and_cache(k, v, torch.zeros(7, 2, 128), torch.zeros(7, 2, 128), slots, "int4")
    with pytest.raises(ValueError):                      # the same tensor without the kind is fp8 of 36 dims
        pa.pa_gather_cache(key, key, k, v, slots)
    with pytest.raises(ValueError):
        pa.pa_gather_cache(key, key.float(), k, v, slots, "int4")
    with pytest.raises(ValueError):
        pa.pa_gather_cache(key, key, k, v, slots.int(), "int4")
    with pytest.raises(ValueError):
        pa.alloc_int4_cache(4, 12, 2, 64, device="cpu")
    assert pa.alloc_int4_cache(4, 8, 2, 64, device="cpu").shape == (4, 8, 2, 36)
    assert not rec.calls


def test_block_bytes(lib):
    assert lib.pa_block_bytes(pa.PA_INT4, 8, 128, 16) == 8 * 16 * 68
    assert lib.pa_block_bytes(pa.PA_INT4, 3, 64, 8) == 3 * 8 * 36
    assert lib.pa_block_bytes(pa.PA_F16, 8, 128, 16) == 8 * 16 * 256
    assert lib.pa_block_bytes(pa.PA_FP8_E5M2, 8, 128, 16) == 8 * 16 * 128
    assert lib.pa_block_bytes(9, 8, 128, 16) == 0 and lib.pa_block_bytes(pa.PA_F16, 0, 128, 16) == 0


W4 = dict(k=16, v=16, kvd=pa.PA_INT4, key=16, val=16, src=pa.PA_F16, slots=16, T=4, Hkv=2, D=128, bs=16, NB=8)


@pytest.mark.parametrize("over,status", [
    (dict(src=pa.PA_INT4), 1),                # a cache type is no element type of a tensor
    (dict(src=pa.PA_FP8_E4M3), 2),
    (dict(D=96), 2),
    (dict(bs=12), 2),
    (dict(slots=None), 1),
    (dict(key=8), 1),
    (dict(T=-1), 1),
    (dict(kvd=6), 1),
])
def test_write_host_validation(lib, over, status):
    a = {**W4, **over}
    assert lib.pa_reshape_and_cache(*(a[x] for x in ("k", "v", "kvd", "key", "val", "src", "slots", "T", "Hkv", "D",
                                                     "bs", "NB")), 1.0, 1.0, None, None) == status
    assert lib.pa_last_error_detail().decode() != ""


@pytest.mark.parametrize("over,status", [
    (dict(src=pa.PA_FP8_E4M3), 2),            # no fp8 destination
    (dict(kvd=pa.PA_F16, src=pa.PA_F32), 2),  # a 16-bit cache gives its own type
    (dict(src=pa.PA_INT4), 1),
    (dict(D=32), 2),
    (dict(bs=4), 2),
    (dict(val=None), 1),
    (dict(val=24), 1),
    (dict(NB=0), 1),
])
def test_gather_host_validation(lib, over, status):
    a = {**W4, **over}
    args = [a[x] for x in ("key", "val", "src", "k", "v", "kvd", "slots", "T", "Hkv", "D", "bs", "NB")]
    assert lib.pa_gather_cache(*args, 1.0, 1.0, None, None) == status
    assert lib.pa_last_error_detail().decode() != ""


def test_gather_refuses_bad_fp8_scales_and_takes_no_tokens(lib):
    args = [16, 16, pa.PA_F16, 16, 16, pa.PA_FP8_E4M3, 16, 4, 2, 128, 16, 8]
    assert lib.pa_gather_cache(*args, 0.0, 1.0, None, None) == 1
    args[7] = 0
    assert lib.pa_gather_cache(*args, 1.0, 1.0, None, None) == 0


def test_attention_binding_reads_4bit_shapes(rec):  # noqa: F811
    k, v = _pool4(D=128)
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    bt, sl = torch.zeros(3, 5, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    pa.pa_decode(torch.empty_like(q), q, k, v, bt, sl, 0.1, "int4")
    a = rec.calls[-1][1]
    assert (a[2], a[5], a[7], a[9], a[10], a[11], a[12], a[13], a[14]) == \
        (pa.PA_BF16, pa.PA_INT4, 5, 3, 4, 2, 128, 16, 10)
    pa.pa_decode_noalloc(torch.empty_like(q), q, k, v, bt, sl, 0.1, "int4")
    assert rec.calls[-1][1][5] == pa.PA_INT4 and rec.calls[-1][1][12] == 128
    qs = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    pa.pa_attention(torch.empty_like(q), q, k, v, bt, sl, qs, 0.1, 2, "int4")
    assert rec.calls[-1][1][5] == pa.PA_INT4 and rec.calls[-1][1][15] == 128
    n = len(rec.calls)
    with pytest.raises(ValueError):
        pa.pa_decode(q[..., :64].contiguous(), q[..., :64].contiguous(), k, v, bt, sl, 0.1, "int4")
    assert len(rec.calls) == n


@pytest.mark.parametrize("over,status", [
    (dict(qd=pa.PA_F32), 2),                   # 16-bit queries
    (dict(qd=pa.PA_INT4), 1),
    (dict(D=96), 2),
    (dict(bs=24), 2),
    (dict(k=8), 1),
    (dict(P=24), 1),
])
def test_int4_decode_host_validation(lib, over, status):
    from test_abi_host import _attention_args, _decode_args
    assert lib.pa_decode(*_decode_args(kvd=pa.PA_INT4, **over)) == status
    assert lib.pa_last_error_detail().decode() != ""
    assert lib.pa_attention(*_attention_args(kvd=pa.PA_INT4, **over)) == status


def test_int4_needs_the_tensor_core_kernel(lib):
    from test_abi_host import _attention_args, _decode_args
    assert lib.pa_decode_simt(*_decode_args(kvd=pa.PA_INT4)) == 2
    assert lib.pa_attention(*_attention_args(kvd=pa.PA_INT4, MQ=65)) == 2      # 130 rows of a KV head
    assert lib.pa_decode(*_decode_args(kvd=pa.PA_INT4, B=0)) == 0
