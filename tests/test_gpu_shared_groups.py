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
