"""The accumulated weights of copied and swapped blocks: the weights pool goes
through the block copies as an f32 pool of head_dim 1."""
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa.build()


@pytest.mark.parametrize("Hkv,bs", [(1, 8), (3, 16), (8, 128)])
def test_weights_follow_their_blocks(Hkv, bs):
    NB = 9
    w = torch.randn(NB, Hkv, bs, device="cuda")
    want = w.clone()
    want[[8, 1]] = want[[0, 7]]
    p = w.view(NB, bs, Hkv, 1)
    pa.pa_copy_blocks(p, p, torch.tensor([[0, 8], [7, 1]], device="cuda"))
    assert torch.equal(w, want)
    host = torch.zeros(4, bs, Hkv, 1).pin_memory()
    pa.pa_swap_blocks(host, host, p, p, torch.tensor([[2, 0], [5, 3]], device="cuda"))
    w[[2, 5]] = float("nan")                          # the blocks' next owner
    pa.pa_swap_blocks(p, p, host, host, torch.tensor([[0, 4], [3, 2]], device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(w[4], want[2]) and torch.equal(w[2], want[5]) and torch.equal(w[[0, 1, 3, 6, 7, 8]], want[[0, 1, 3, 6, 7, 8]])


def test_a_preempted_request_evicts_as_if_it_had_stayed():
    """Weights added up, the request swapped out and in to other blocks, then evicted."""
    g = torch.Generator().manual_seed(9)
    NB, bs, Hkv, D, L = 40, 16, 2, 64, 230
    k, v = (torch.randn(NB, bs, Hkv, D, generator=g).half().cuda() for _ in range(2))
    w = torch.zeros(NB, Hkv, bs, device="cuda")
    q = torch.randn(1, 8, D, generator=g).half().cuda()
    old = torch.arange(15, dtype=torch.int32, device="cuda").view(1, -1)
    new = torch.arange(39, 24, -1, dtype=torch.int32, device="cuda").view(1, -1)
    sl = torch.tensor([L], dtype=torch.int32, device="cuda")
    out, kept = torch.empty_like(q), [torch.empty(1, Hkv, 64, dtype=torch.int32, device="cuda") for _ in range(2)]
    pa.pa_decode_weights(out, w, q, k, v, old, sl, 0.125, fresh=sl)
    hk, hv = (torch.zeros(15, bs, Hkv, D, dtype=torch.float16).pin_memory() for _ in range(2))
    hw, p = torch.zeros(15, bs, Hkv, 1).pin_memory(), w.view(NB, bs, Hkv, 1)
    away = torch.stack([old[0], torch.arange(15, device="cuda")], 1).long()
    back = torch.stack([torch.arange(15, device="cuda"), new[0]], 1).long()
    for a, b, m in ((hk, k, 0), (hw, p, 1)):
        x, y = (hv, v) if m == 0 else (a, b)
        pa.pa_swap_blocks(a, x, b, y, away)
        pa.pa_swap_blocks(b, y, a, x, back)
    for t, r in ((new, kept[0]), (old, kept[1])):
        pa.pa_evict(k, v, w, t, sl, torch.empty_like(sl), 64, num_sink=2, num_recent=8, kept=r)
    assert torch.equal(kept[0], kept[1]) and kept[0].min() >= 0
    n = 64 // bs
    assert torch.equal(k[new[0, :n].long()], k[old[0, :n].long()]) and torch.equal(w[new[0, :n].long()], w[old[0, :n].long()])
