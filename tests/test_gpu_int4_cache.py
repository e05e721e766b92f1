"""4-bit pools on the GPU: writes bit for bit against the definition in 64
bits, reads against the values, block copies and swaps as bytes."""
import numpy as np
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _int4

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SMALLEST = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}    # half the spacing next to zero


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa.build()


def _write(x, y, slots, NB, bs, fill=0xA5):
    T, Hkv, D = x.shape
    k = torch.full((NB, bs, Hkv, D // 2 + 4), fill, dtype=torch.uint8, device="cuda")
    v = torch.full_like(k, fill)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_reshape_and_cache(k, v, x.cuda(), y.cuda(), slots.cuda(), "int4", err_flag=err)
    torch.cuda.synchronize()
    return k, v, int(err.item())


def _want(x, slots, NB, bs, fill=0xA5):
    """The pool after the write, from the definition."""
    T, Hkv, D = x.shape
    pool = np.full((NB, bs, Hkv, D // 2 + 4), fill, np.uint8)
    code, step, low = _int4.encode(x.double().numpy())
    c, s, lo = _int4.rows(pool)
    for t, sl in enumerate(slots.tolist()):
        if 0 <= sl < NB * bs:
            c[sl // bs, sl % bs], s[sl // bs, sl % bs], lo[sl // bs, sl % bs] = code[t], step[t], low[t]
    return _int4.pack(c, s, lo)


def _same_pool(got, want):
    """Equal bits, except that any two NaN parameters are equal."""
    gc, gp = _int4.split(got.cpu().numpy())
    wc, wp = _int4.split(want)
    assert (gc == wc).all()
    nan = np.isnan(wp)
    assert (np.isnan(gp) == nan).all()
    assert (gp.view(np.uint16)[~nan] == wp.view(np.uint16)[~nan]).all()


def _special_rows(D, dtype, gen):
    """Rows where quantising can go wrong."""
    r = torch.randn(16, D, generator=gen)
    r[0] = 0.0
    r[1] = -3.7
    r[2] = torch.arange(D) % 31 / 2.0                      # low 0, step 1: every other quotient is a half
    r[3] *= 1e-6                                           # step below the smallest normal f16
    r[4] *= 1e-9                                           # step rounds to zero
    r[5, 3] = float("inf")
    r[6, 1] = -float("inf")
    r[7, D - 1] = float("nan")
    r[8] = 1e30 * torch.sign(r[8])
    r[9] = torch.where(torch.arange(D) % 2 == 0, 65504.0, -65504.0)
    r[10] = 1.0
    r[10, 5] = 1.0 + 2.0 ** -7                             # one value off a constant row
    r[11] = -torch.arange(D).float()
    r[12] *= 1e4
    r[13] = 1000.0 + r[13] * 1e-2                          # a mean far above the spread: low itself is rounded
    r[14] = -1000.0 + r[14] * 1e-2
    r[15, 2] = 300.0                                       # an outlier
    return r.to(DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,Hkv,D,bs", [(1, 1, 128, 8), (33, 3, 64, 16), (257, 8, 128, 32), (130, 5, 64, 128),
                                        (97, 2, 128, 24)])
def test_write_equals_the_definition(dtype, T, Hkv, D, bs):
    g = torch.Generator().manual_seed(T * 7 + D)
    x = (torch.randn(T, Hkv, D, generator=g) + torch.randn(Hkv, D, generator=g)).to(DT[dtype])
    y = (torch.randn(T, Hkv, D, generator=g) * 10.0 ** (torch.rand(T, Hkv, 1, generator=g) * 7 - 4)).to(DT[dtype])
    sp = _special_rows(D, dtype, g)
    n = min(T * Hkv, 16)
    y.view(-1, D)[:n] = sp[:n]
    x.view(-1, D)[-n:] = sp[-n:]
    NB = -(-T // bs) + 2
    slots = torch.randperm(NB * bs, generator=g)[:T]
    if T > 20:
        slots[3], slots[17] = -1, -5                        # padding: skipped
    k, v, err = _write(x, y, slots, NB, bs)
    assert err == 0
    _same_pool(k, _want(x, slots, NB, bs))
    _same_pool(v, _want(y, slots, NB, bs))


def test_write_of_many_random_rows_has_no_code_off():
    """Every code of 60,000 f32 rows: the comparisons at the middle between two values are exact."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(15000, 4, 64, generator=g)
    slots = torch.randperm(15008, generator=g)[:15000]
    k, v, err = _write(x, -x, slots, 15008 // 16, 16, 0)
    for got, src in ((k, x), (v, -x)):
        code, step, low = _int4.encode(src.double().numpy())
        c, s, lo = (a.reshape((-1,) + a.shape[2:])[slots.numpy()] for a in _int4.rows(got.cpu().numpy()))
        assert (s.view(np.uint16) == step.view(np.uint16)).all() and (lo == low).all() and (c == code).all()


def test_bad_slots_are_flagged_and_skipped():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(9, 2, 64, generator=g).half()
    slots = torch.tensor([0, 5, 48, 7, 1 << 40, 47, -1, 12, 13])
    k, v, err = _write(x, x, slots, 3, 16)
    assert err == pa.ERRBIT_BAD_SLOT
    _same_pool(k, _want(x, slots, 3, 16))
    out = torch.full((9, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    out2 = out.clone()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_gather_cache(out, out2, k, v, slots.cuda(), "int4", err_flag=flag)
    assert flag.item() == pa.ERRBIT_BAD_SLOT
    for t in (2, 4, 6):
        assert (out[t] == 7.0).all() and (out2[t] == 7.0).all()      # left as they were
    assert not (out[0] == 7.0).all()


@pytest.mark.parametrize("dst", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Hkv,D,bs", [(1, 64, 8), (4, 128, 16), (3, 128, 40)])
def test_gather_gives_the_values(dst, Hkv, D, bs):
    rng = np.random.default_rng(D + Hkv)
    NB, T = 7, 75
    code = rng.integers(0, 16, (NB, bs, Hkv, D)).astype(np.uint8)
    par = []
    for _ in range(2):
        step = np.abs(rng.standard_normal((NB, bs, Hkv)) * 10.0 ** rng.uniform(-6, 3, (NB, bs, Hkv))).astype(np.float16)
        low = (rng.standard_normal((NB, bs, Hkv)) * 10.0 ** rng.uniform(-3, 3, (NB, bs, Hkv))).astype(np.float16)
        step[0, 0, 0], low[0, 1, 0] = 0, np.float16("nan")
        par.append((step, low))
    pools = [torch.from_numpy(_int4.pack(code, *p)).cuda() for p in par]
    slots = rng.integers(0, NB * bs, T)
    slots[:4] = (0, 1, 1, NB * bs - 1)                     # a slot twice, the last one
    out = [torch.empty(T, Hkv, D, dtype=DT[dst], device="cuda") for _ in range(2)]
    pa.pa_gather_cache(out[0], out[1], pools[0], pools[1], torch.from_numpy(slots).cuda(), "int4")
    for o, p in zip(out, par):
        want = _int4.decode(code, *p).reshape(NB * bs, Hkv, D)[slots]
        got = o.double().cpu().numpy()
        assert (np.isnan(got) == np.isnan(want)).all()
        ok = ~np.isnan(want)
        # rounded to f32, then to the type: half a step of each
        rel = HALF_STEP[dst] + (0 if dst == "f32" else HALF_STEP["f32"] * 1.01)
        assert (np.abs(got - want)[ok] <= rel * np.abs(want[ok]) + SMALLEST[dst]).all()


@pytest.mark.parametrize("kv,dst", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("fp8_e4m3", "f16"),
                                    ("fp8_e4m3", "f32"), ("fp8_e5m2", "bf16")])
def test_gather_of_other_caches(kv, dst):
    g = torch.Generator().manual_seed(8)
    NB, bs, Hkv, D = 6, 16, 3, 64
    slots = torch.randperm(NB * bs, generator=g)[:50]
    out = [torch.empty(50, Hkv, D, dtype=DT[dst], device="cuda") for _ in range(2)]
    if kv in DT:
        pools = [torch.randn(NB, bs, Hkv, D, generator=g).to(DT[kv]) for _ in range(2)]
        want = [p.view(-1, Hkv, D)[slots].double().numpy() for p in pools]
        pools = [p.cuda() for p in pools]
    else:
        st = torch.uint8 if kv == "fp8_e4m3" else torch.float8_e5m2
        by = [torch.randint(0, 256, (NB, bs, Hkv, D), generator=g, dtype=torch.uint8) & 0xBB for _ in range(2)]
        f8 = torch.float8_e4m3fn if kv == "fp8_e4m3" else torch.float8_e5m2
        want = [b.view(f8).double().view(-1, Hkv, D)[slots].numpy() * s for b, s in zip(by, (0.5, 0.37))]
        pools = [b.view(st).cuda() for b in by]
    pa.pa_gather_cache(out[0], out[1], pools[0], pools[1], slots.cuda(), k_scale=0.5, v_scale=0.37)
    for o, w in zip(out, want):
        got = o.double().cpu().numpy()
        if kv in DT:
            assert (got == w).all()
        else:
            # the scale is an f32 number, the product is rounded to f32, then to the type
            rel = 2 * HALF_STEP["f32"] + HALF_STEP[dst] * 1.01
            assert (np.abs(got - w) <= rel * np.abs(w) + SMALLEST[dst]).all()


def test_block_copies_and_swaps_move_4bit_blocks():
    g = torch.Generator().manual_seed(6)
    NB, bs, Hkv, D = 9, 16, 3, 64
    k = torch.randint(0, 256, (NB, bs, Hkv, D // 2 + 4), generator=g, dtype=torch.uint8)
    v = torch.randint(0, 256, k.shape, generator=g, dtype=torch.uint8)
    pairs = torch.tensor([[0, 8], [7, 1], [3, 4]])
    want = [x.clone() for x in (k, v)]
    for w in want:
        w[pairs[:, 1]] = w[pairs[:, 0]]
    kd, vd = k.cuda(), v.cuda()
    pa.pa_copy_blocks(kd, vd, pairs.cuda(), "int4")
    assert torch.equal(kd.cpu(), want[0]) and torch.equal(vd.cpu(), want[1])
    layers = [(k.cuda(), v.cuda()) for _ in range(3)]
    pa.pa_copy_blocks_layers([a for a, _ in layers], [b for _, b in layers], pairs.cuda(), "int4")
    for a, b in layers:
        assert torch.equal(a.cpu(), want[0]) and torch.equal(b.cpu(), want[1])
    hk, hv = (torch.zeros(4, bs, Hkv, D // 2 + 4, dtype=torch.uint8).pin_memory() for _ in range(2))
    out = torch.tensor([[2, 0], [5, 3]]).cuda()
    pa.pa_swap_blocks(hk, hv, kd, vd, out, "int4")
    torch.cuda.synchronize()
    assert torch.equal(hk[0], want[0][2]) and torch.equal(hk[3], want[0][5]) and torch.equal(hv[3], want[1][5])
    assert not hk[1].any()


def test_write_and_gather_on_another_stream_and_in_a_graph():
    g = torch.Generator().manual_seed(7)
    x = torch.randn(40, 2, 128, generator=g).bfloat16().cuda()
    slots = torch.randperm(48, generator=g)[:40].cuda()
    k = pa.alloc_int4_cache(3, 16, 2, 128)
    v, out, out2 = torch.zeros_like(k), torch.empty_like(x), torch.empty_like(x)

    def both():
        pa.pa_reshape_and_cache(k, v, x, x, slots, "int4")
        pa.pa_gather_cache(out, out2, k, v, slots, "int4")

    both()
    torch.cuda.synchronize()
    ref = out.clone()
    s = torch.cuda.Stream()
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        k.zero_()
        both()
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(out2, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    out.zero_()
    k.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
