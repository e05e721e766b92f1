"""Groups of pa_decode_shared that do not fit: their sequences attend by themselves, whatever
their prefixes say, and the other groups are as ever."""
import pytest
import torch

import paged_kv_cache_69_gb300 as pa

import _prompt as ref
from test_gpu_shared import F16, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("starts,prefix", [([0, 4, 9], [900, 5000]), ([0, 4, 9], [900, 2 ** 31 - 1]), ([-1, 4, 6], [5000, 2100]),
                                           ([-2 ** 31, 4, 6], [1100, 2100]), ([0, 4, 2 ** 31 - 1], [900, 2200])])
def test_prefixes_of_groups_that_leave_the_batch(starts, prefix):
    """...are longer than their sequences."""
    c = Case([(900, [5, 6, 7, 8]), (2100, [9, 10])], 16, 2, 64, F16, spare=400)
    fill = torch.full((6, 400), -1, dtype=torch.int32, device="cuda")                # tables that such a prefix would fit
    c.tables = torch.cat([c.tables, fill], 1).contiguous()
    want = c.want()
    c.starts, c.prefix = c.dev(starts), c.dev(prefix)
    out = c.call()
    assert c.err.item() == pa.ERRBIT_BAD_QUERY
    ref.check(out, *want)


@pytest.mark.parametrize("starts,prefix", [([0, 200, 100, 240], [1024, 0, 512]), ([0, 200, 100, 240], [512, 0, 1024]),
                                           ([30, 240, 0, 100, 90, 240], [1024, 0, 1008, 0, 560]),
                                           ([0, 240, 0, 240, 0, 240, 0, 240], [1024, 0, 512, 0, 256, 0, 1024])])
def test_groups_that_overlap(starts, prefix):
    """Entries that fall back: what lies between belongs to two groups that fit, and is attended with one of them."""
    c = Case([(1024, [1 + i % 40 for i in range(240)])], 16, 2, 64, F16)
    want = c.want()
    c.starts, c.prefix = c.dev(starts), c.dev(prefix)
    out = c.call()
    assert c.err.item() == pa.ERRBIT_BAD_QUERY
    ref.check(out, *want)


def test_many_small_groups():
    """Groups of one and two beside large ones, more of them than CTAs."""
    g = torch.Generator().manual_seed(8)
    n = [1 + int(x) for x in torch.randint(0, 2, (330,), generator=g)] + [70, 33]
    c = Case([(2100 if m == 2 and i % 40 == 0 else 40 * (m > 2) * 16, [1 + (i + j) % 5 for j in range(m)]) for i, m in enumerate(n)],
             8, 2, 64, F16)
    c.check(c.call())


def test_more_groups_than_the_scheduler_keeps():
    c = Case([(16 * (i % 3), [1 + i % 7]) for i in range(1300)] + [(1024, [1, 2, 3, 40])] + [(0, [2])] * 50 + [(2048, [5, 6])], 4, 2, 64, F16)
    c.check(c.call())


@pytest.mark.parametrize("groups", [0, 1, 16, 256, 1024])
def test_workspace_grows_with_rows_and_not_with_groups(groups):
    """Beside what pa_decode takes: a partial per (sequence, head), and those of prefixes cut into ranges
    to fill the GPU, two per SM of 256 rows each."""
    B, Hq, Hkv, D = 1024, 32, 8, 128
    base = pa.pa_decode_workspace_size(B, Hq, 8192, D, 0)
    more = pa.pa_decode_shared_workspace_size(B, groups, Hq, Hkv, 8192, D) - base
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert 0 < more <= (B * Hq + 2 * sms * 256) * (D * 4 + 8) + (1 << 16)
    few = pa.pa_decode_shared_workspace_size(2, 1, 4, 2, 8192, 64) - pa.pa_decode_workspace_size(2, 4, 8192, 64, 0)
    assert few <= 32 * 2 * 4 * (64 * 4 + 8) + (1 << 16)
