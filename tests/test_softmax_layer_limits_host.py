"""Softmax-layer operators without a GPU: refusals and builds at the edges of
their contracts."""
import pytest

import lightning_attention_attn_gb300 as la
from lightning_attention_attn_gb300 import build as labuild

A = 0x100000  # an aligned fake address: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    return la.load(labuild.build())


@pytest.mark.parametrize("lens_out, count_out", [(A, A + 0x100), (A + 0x100, A)])
def test_paged_reserve_refuses_new_lens_as_an_output(lib, lens_out, count_out):
    a = 2 * A
    status = lib.lightning_attn_paged_reserve(a, 5, 5, a, A, None, 4, a, a, 10, 16, 4, a, a, a, a,
                                              lens_out, count_out, None)
    assert status == la.LA_ERR_INVALID_ARG
    assert "new_lens" in lib.lightning_attn_last_error().decode()
