"""The bounded waits of the block-scaled decode, made to run out on purpose.

The testing hook makes each warp wait, with its first copies in flight, on a barrier
that nothing completes, for at most 2 ms: the warp records code 1, starts no further
copies, meets its block's and cluster's barriers, waits for its copies in flight and
returns. Nothing faults and no wait is unbounded. The next call is correct again, with
a clean error word."""
import pytest
import torch

import attention_learned_sinks_gb300 as sa
from helpers import check_close
from test_parity_block_cache import Case

pytestmark = pytest.mark.gpu

STALL_NS = 2_000_000


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,num_splits", [([900, 50, 1200, 0], 1), ([900, 50, 1200, 0], 5),
                                             ([9000, 50, 3000, 0, 7], 17),
                                             ([100, 50, 128] * 440, 0)])
def test_decode_timeout_path_then_recovers(lens, num_splits, d):
    c = Case(lens, 8, 2, d, 16, 16, seed=97)
    torch.cuda.synchronize()
    assert sa.sinkattn_get_device_error() == 0
    sa.sinkattn_debug_stall_waits(STALL_NS)
    try:
        c.decode(num_splits)
        torch.cuda.synchronize()
    finally:
        sa.sinkattn_debug_stall_waits(0)
    assert sa.sinkattn_get_device_error() == 1
    out, lse = c.decode(num_splits)
    check_close(out, lse, *c.reference(), "decode after a timed-out call", c.vmax)
    assert sa.sinkattn_get_device_error() == 0


def test_layouts_without_barriers_do_not_wait():
    c = Case([900, 50, 1200], 8, 2, 64, 24, 8, seed=98)
    sa.sinkattn_debug_stall_waits(STALL_NS)
    try:
        out, lse = c.decode()
        torch.cuda.synchronize()
    finally:
        sa.sinkattn_debug_stall_waits(0)
    check_close(out, lse, *c.reference(), "decode without barriers", c.vmax)
    assert sa.sinkattn_get_device_error() == 0
