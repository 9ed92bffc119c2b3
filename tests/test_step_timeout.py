"""The tree attention's bounded waits: a wait that runs out records code 1, every CTA
ends, and the next call is right."""
import pytest
import torch

import attention_learned_sinks_gb300 as sa
from test_parity_step import Tree

pytestmark = pytest.mark.gpu

STALL_NS = 2_000_000


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,old,splits", [([5, 17, 1, 0], [1500, 300, 20, 7], 0),
                                            ([5, 17, 1, 0], [1500, 300, 20, 7], 1),
                                            ([4] * 400, [60] * 400, 0)])
def test_tree_timeout_path_then_recovers(new, old, splits, d):
    t = Tree(new, old, 16, 8, 2, d)
    a, kw = t.args(), t.kw()
    torch.cuda.synchronize()
    assert sa.sinkattn_get_device_error() == 0
    sa.sinkattn_debug_stall_waits(STALL_NS)
    try:
        sa.sinkattn_decode_tree(*a, **kw, num_splits=splits)
        torch.cuda.synchronize()
    finally:
        sa.sinkattn_debug_stall_waits(0)
    assert sa.sinkattn_get_device_error() == 1
    t.check("tree attention after a timed-out call", num_splits=splits)
