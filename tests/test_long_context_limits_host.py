"""The long-context operators of the softmax layers at the limits of their contract, without a GPU."""
import os

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


# ----------------------------------------- outputs that a call still reads
# bf16, 4 tokens, 8 query and 2 key-value heads of 64; every array in a place of its own
AT = {n: A * (i + 1) for i, n in enumerate("q bd pt pl kc vc bt lens sel out ws".split())}


def _call(lib, name, at, stride=512, batch=4):
    p = {**AT, **{n: AT[o] for n, o in at.items()}}
    q, shape = [p["q"], stride], [batch, 8, 2, 64, la.LA_DTYPE_BF16]
    cache, table, pool = [p["kc"], 2048, p["vc"], 2048], [p["bt"], 5, 5, p["lens"]], [10, 16]
    end = [0.1, p["out"], None, p["ws"], 0, None]  # a workspace that is too small: nothing is launched
    args = {"paged_decode": q + cache + table + pool + shape + end,
            "paged_sparse_decode": q + cache + table + [p["sel"], 3] + pool + shape + end,
            "paged_prefix_decode": q + cache + [p["pt"], 5, p["pl"]] + table + pool + shape + end,
            "paged_select": q + [p["bd"], 256] + table + pool + shape + [3, 1, 1, p["sel"], p["ws"], 0, None]}[name]
    status = getattr(lib, "lightning_attn_" + name)(*args)
    assert status == BAD
    return lib.lightning_attn_last_error().decode()


@pytest.mark.parametrize("name, at", [("paged_select", dict(sel="bt")), ("paged_select", dict(sel="lens"))])
def test_outputs_over_other_arguments_are_refused(lib, name, at):
    assert " one array" in _call(lib, name, at) and "workspace too small" in _call(lib, name, {})


@pytest.mark.parametrize("name", ["paged_decode", "paged_sparse_decode", "paged_prefix_decode"])
def test_an_output_in_place_of_strided_queries_is_refused(lib, name):
    """Its rows would lie over queries of other requests that have not been read."""
    assert "in place" in _call(lib, name, dict(out="q"), stride=520)
    for ok in (_call(lib, name, dict(out="q")), _call(lib, name, dict(out="q"), stride=520, batch=1),
               _call(lib, name, {}, stride=520)):
        assert "workspace too small" in ok


# ------------------------------------------------------------------- contract
def test_contract_names_every_kernel_whose_waits_may_give_up():
    """The calls whose device error words device_status takes are named there, and send their caller to it."""
    with open(os.path.join(labuild.ROOT, "include", "lightning_attn.h")) as f:
        header = f.read()

    def before(entry):  # the comment in front of a declaration
        at = header.index("la_status lightning_attn_" + entry + "(")
        return header[header.rindex("/*", 0, at):at]

    assert "prefill" in before("device_status") and "prefix" in before("device_status")
    assert "lightning_attn_device_status" in before("paged_prefix_decode")
    assert "device_status" in la.paged_prefix_decode.__doc__
