"""Graphs captured once and replayed while sequences grow, end, begin in other
blocks and are evicted, as a server replays its step: every replay equals an
eager call on the same tensors."""
import numpy as np
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

pytestmark = pytest.mark.gpu

B, Hq, Hkv, D, BS, NB, MB = 4, 8, 2, 128, 16, 700, 160


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa.build()


class Server:
    def __init__(self, kv, seed):
        g = torch.Generator().manual_seed(seed)
        x = [torch.randn(NB * BS, Hkv, D, generator=g).half().cuda() for _ in range(2)]
        if kv == "int4":
            self.k, self.v = pa.alloc_int4_cache(NB, BS, Hkv, D), pa.alloc_int4_cache(NB, BS, Hkv, D)
        else:
            self.k, self.v = (torch.zeros(NB, BS, Hkv, D, dtype=torch.float16, device="cuda") for _ in range(2))
        self.kv = kv
        pa.pa_reshape_and_cache(self.k, self.v, *x, torch.arange(NB * BS, device="cuda"), kv if kv == "int4" else None)
        self.w = torch.rand(NB, Hkv, BS, generator=g).cuda()
        self.q = torch.randn(B, Hq, D, generator=g).half().cuda()
        self.bt = torch.full((B, MB), -1, dtype=torch.int32, device="cuda")
        self.sl = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.fresh = torch.ones(B, dtype=torch.int32, device="cuda")
        self.out = torch.zeros_like(self.q)
        self.kept = torch.zeros(B, Hkv, 300, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (
            pa.pa_decode_weights_workspace_size(B, Hq, MB * BS, D), pa.pa_evict_workspace_size(B, Hkv, MB * BS, 300))]

    def step(self):
        pa.pa_decode_weights(self.out, self.w, self.q, self.k, self.v, self.bt, self.sl, 0.09, self.kv,
                             fresh=self.fresh, workspace=self.ws[0], err_flag=self.err)
        pa.pa_evict(self.k, self.v, self.w, self.bt, self.sl, self.sl, 300, self.kv, num_sink=4, num_recent=32,
                    kept=self.kept, workspace=self.ws[1], err_flag=self.err)

    def set(self, lens, rng):
        order, first = rng.permutation(NB), 0
        t = np.full((B, MB), -1, np.int32)
        for i, L in enumerate(lens):
            n = -(-L // BS)
            t[i, :n] = order[first:first + n]
            first += n
        self.bt.copy_(torch.from_numpy(t))
        self.sl.copy_(torch.tensor(lens, dtype=torch.int32))
        self.fresh.copy_(torch.tensor([min(L, 3) for L in lens], dtype=torch.int32))

    def state(self):
        return [x.clone() for x in (self.out, self.w, self.k, self.v, self.sl, self.kept, self.err)]


@pytest.mark.parametrize("kv", ["int4", "f16"])
def test_a_replay_takes_the_lengths_it_finds(kv):
    a, b = Server(kv, 5), Server(kv, 5)
    rng = [np.random.default_rng(6) for _ in range(2)]
    for s, r in zip((a, b), rng):
        s.set([1, 2, 3, 4], r)
    b.step()
    a.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    for lens in ([300, 301, 0, 2560], [0, 0, 0, 0], [17, 1, 2559, 299], [0, 0, 2000, 0], [2400, 2500, 2501, 2560],
                 [1, 0, 0, 0]):
        for s, r in zip((a, b), rng):
            s.set(lens, r)
        a.step()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y)
        assert a.err.item() == 0 and a.sl.tolist() == [min(L, 300) for L in lens]
        assert torch.isfinite(a.out).all() and torch.isfinite(a.w).all()
        for i, L in enumerate(lens):
            assert bool(a.out[i].any()) == (L > 0)
