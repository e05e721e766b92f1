"""The merge of cut prompt items takes the places of its partials from the workspace, where
a launch leaves them.  A launch whose wait ran out may leave any of them unwritten, so that
they hold what was there before: such entries lead to no read or write outside the call's
buffers, and the entries beside them are merged as ever."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

from paged_kv_cache_69_gb300 import build_lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_cache_69_gb300", "csrc")
INT = 2 ** 31


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("mergeprobe") / "libmergeprobe.so")
    cmd = [build_lib._nvcc(), *build_lib.NVCC_FLAGS, "-shared", f"-I{CSRC}", os.path.join(ROOT, "tests", "gpu_merge_probe.cu"),
           "-o", out, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(out)
    lib.merge_parts.argtypes = [ctypes.c_int] * 5 + [ctypes.POINTER(ctypes.c_int)] * 2
    lib.merge_run.argtypes = [ctypes.c_void_p] * 4 + [ctypes.c_int] * 4
    return lib


def _parts(probe, Hq, Hkv, total_q, grid, i, n, item):
    ints = lambda x: (ctypes.c_int * 4)(*x)  # noqa: E731
    return probe.merge_parts(Hq, Hkv, total_q, grid, i, ints(n), ints(item))


def test_entries_of_a_launch(probe):
    """Spans of a / b items: item i has part in spans floor(i b / a) to ceil((i + 1) b / a) - 1."""
    for b, a, items in ((2, 1, 70), (32, 1, 4), (3, 2, 100), (9, 7, 118), (32, 31, 147)):
        for i in range(items):
            first, end = i * b // a, -(-(i + 1) * b // a)
            got = _parts(probe, 28, 4, 36 * items, 152, i, (b, items, a, 0), (36 * i, 36, i % 4, first + i))
            assert got == end - first and 1 <= got <= 32
        assert _parts(probe, 28, 4, 36 * items, 152, items, (b, items, a, 0), (0, 36, 0, 0)) == 0
    assert _parts(probe, 28, 4, 5000, 152, 0, (1, 0, 1, 0), (0, 36, 0, 0)) == 0          # nothing was cut


def test_entries_that_cannot_be_ones(probe):
    good = ((4, 10, 3, 0), (100, 36, 3, 20))
    assert _parts(probe, 28, 4, 500, 20, 5, *good) == 2
    for at, field, values in ((0, 0, (-INT, -4, 0, 1, 3, 33, INT - 1)), (0, 1, (-INT, 0, 5)), (0, 2, (-INT, -1, 0, 4, INT - 1)),
                              (1, 0, (-INT, -1, 465, INT - 1)), (1, 1, (-INT, 0, 37, INT - 1)), (1, 2, (-INT, -1, 4, INT - 1)),
                              (1, 3, (-INT, -1, 39, INT - 1))):
        for x in values:
            e = [list(y) for y in good]
            e[at][field] = x
            assert _parts(probe, 28, 4, 500, 20, 5, *e) == 0, (at, field, x)


def test_whatever_the_workspace_holds(probe):
    """Accepted entries stay within the rows, the heads and the places, whatever they hold."""
    r = random.Random(1)
    near = lambda top: r.randrange(-2, top + 3) if r.random() < 0.9 else r.randrange(-INT, INT)  # noqa: E731
    taken = 0
    for _ in range(20000):
        Hkv = r.choice([1, 2, 8])
        G, total_q, grid = r.choice([1, 3, 7, 128]), r.choice([1, 40, 5000, (1 << 30) - 1]), r.choice([1, 20, 152])
        n = [near(32), near(grid), near(32), 0]
        item, i = [near(total_q), near(2 * (128 // G)), near(Hkv), near(2 * grid)], r.randrange(grid)
        parts = _parts(probe, G * Hkv, Hkv, total_q, grid, i, n, item)
        assert 0 <= parts <= 32
        if parts:
            taken += 1
            assert 0 <= item[0] and item[0] + item[1] <= total_q and 1 <= item[1] <= 2 * (128 // G)
            assert 0 <= item[2] < Hkv and 0 <= item[3] and item[3] + parts <= 2 * grid
    assert taken > 50


@pytest.mark.gpu
def test_merge_beside_entries_that_were_never_written(probe):
    Hq, Hkv, D, T, grid, G, tokens = 4, 2, 64, 300, 6, 2, 64
    g = torch.Generator().manual_seed(4)
    acc, ml = torch.randn(2 * grid, 2, 128, D, generator=g).cuda(), torch.rand(2 * grid, 2, 128, 2, generator=g).cuda() + 0.5
    # items 0, 2 and 4 are whole entries of three spans each, the rest is what a workspace may hold
    whole = {0: (0, 128, 1, 0), 2: (130, 70, 0, 4), 4: (299, 1, 1, 9)}
    cut = torch.full((1 + grid, 4), INT - 1, dtype=torch.int32)
    cut[0] = torch.tensor([3, grid, 1, 0])
    cut[2], cut[4], cut[6] = torch.tensor([280, 128, 0, 0]), torch.tensor([-7, 128, 1, 3]), torch.tensor([0, 128, 1, 10])
    for i, e in whole.items():
        cut[1 + i] = torch.tensor(e)
    out = torch.full((64 + T * Hq * D + 64,), 7.0, dtype=torch.float16, device="cuda")
    want = torch.full((T, Hq, D), 7.0, dtype=torch.float64, device="cuda")
    for row0, n, h, place in whole.values():
        a, m = acc[place:place + 3].double(), ml[place:place + 3].double()
        w = torch.exp2(m[..., 0] - m[..., 0].amax(0))
        o = (w[..., None] * a).sum(0) / (w * m[..., 1]).sum(0)[..., None]
        o = o.view(2, tokens, G, D).reshape(2 * tokens, G, D)                   # tile row u: token u / G, head u % G
        want[row0:row0 + n, h * G:(h + 1) * G] = o[:n]
    assert probe.merge_run(out[64:].data_ptr(), cut.cuda().data_ptr(), ml.data_ptr(), acc.data_ptr(), Hq, Hkv, T, grid) == 0
    got = out[64:-64].view(T, Hq, D).double()
    # one rounding to f16; sums of three terms, exponentials (2^-22 each) and a quotient in f32: under
    # 2^-20 of sum w |acc| / sum w l <= 5 / 0.5
    assert ((got - want).abs() <= want.abs() * 2.0 ** -11 + 2.0 ** -16).all()
    assert (out[:64] == 7).all() and (out[-64:] == 7).all()
    # no entry at all
    out.fill_(7)
    for first in ([INT - 1] * 4, [-1] * 4, [32, INT - 1, 1, 0], [0, grid, 0, 0]):
        cut = torch.full((1 + grid, 4), -INT, dtype=torch.int32)
        cut[0] = torch.tensor(first)
        cut = cut.cuda()
        assert probe.merge_run(out[64:].data_ptr(), cut.data_ptr(), ml.data_ptr(), acc.data_ptr(), Hq, Hkv, T, grid) == 0
        assert (out == 7).all()
