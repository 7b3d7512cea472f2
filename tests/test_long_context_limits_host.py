"""The long-context operators of the softmax layers at the limits of their contract, without a GPU."""
import pytest

import lightning_attention_attn_gb300 as la
from lightning_attention_attn_gb300 import build as labuild

A = 0x100000  # an aligned fake address: validation fails before any use
BAD = la.LA_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    return la.load(labuild.build())


@pytest.mark.parametrize("width", [2 ** 31 - 1, 2 ** 30, 200000])
@pytest.mark.parametrize("batch, heads", [(1, 1), (1, 2), (3, 1), (128, 8)])
def test_select_steps_stay_within_32_bits(lib, batch, heads, width):
    """Scores of a unit's blocks (at most 2^31 - 2^16) are taken by some warps, 16 blocks each in turn, a turn
    ahead: the index behind the last block still fits 32 bits.  The workspace holds 12 bytes a block and 4 a warp."""
    size = lib.lightning_attn_paged_select_workspace_bytes(batch, heads, width)
    warps = -(-(size - 12 * batch * heads * width) // (4 * batch * heads))
    assert 1 <= warps and (2 ** 31 - 2 ** 16) + 16 * warps + 16 < 2 ** 31
