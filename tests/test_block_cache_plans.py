"""Host-side plans of the block-scaled cache's calls (no GPU): scratch that they ask for."""
import pytest

import attention_learned_sinks_gb300 as sa
from attention_learned_sinks_gb300 import build as sbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    sbuild.build()


@pytest.mark.parametrize("d,most", [(64, 304), (128, 228)])
def test_even_shares_have_the_limits_that_the_header_states(d, most):
    """num_splits above 16 shares the keys out (partials, so scratch) for up to 4096
    sequences and up to half of the resident blocks' number of heads; else it does not."""
    size = sa.sinkattn_decode_fp8_block_workspace_size
    assert size(2, 64000, most, most, d, num_splits=17) > 0
    assert size(2, 64000, most + 1, most + 1, d, num_splits=17) == 0
    assert size(4096, 64000, 8, 1, d, num_splits=17) > 0
    assert size(4097, 64000, 8, 1, d, num_splits=17) == 0
    # tiles of 8 query heads count like KV heads
    assert size(2, 64000, 16 * most, most, d, num_splits=17) == 0
    assert size(2, 64000, 8, 1, d, num_splits=17) == size(2, 64000, 8, 1, d, num_splits=1000)


def test_prefill_scratch_holds_a_factor_per_sequence_and_head():
    args = (100, 5000, 64, 700, 16, 8, 64, 0, 1)
    block = sa.sinkattn_prefill_paged_fp8_block_workspace_size(*args)
    plain = sa.sinkattn_prefill_paged_workspace_size(*args)
    assert block >= plain + 100 * 8 * 4 and block % 256 == plain % 256 == 0
