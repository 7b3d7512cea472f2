"""The long-context operators of the softmax layers without a GPU: the reference checks itself, and
library and binding refuse bad calls before anything is launched."""
import pytest
import torch

import long_context_reference as lref
import softmax_reference as ref
import lightning_attention_attn_gb300 as la
from lightning_attention_attn_gb300 import build as labuild

A = 0x100000  # an aligned fake address: validation fails before any use
BAD = la.LA_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    return la.load(labuild.build())


# --------------------------------------------------------------- reference
def test_reference_scores_bound_every_product():
    g = torch.Generator().manual_seed(1)
    pages, kv, page, d = 6, 2, 5, 8
    kc = torch.randn(pages, kv, page, d, generator=g)
    bt = torch.tensor([[3, 0, 5]], dtype=torch.int32)
    bd = lref.bounds(kc, torch.zeros(pages, kv, 2, d), bt, [0], [13])
    assert (bd[[1, 2, 4]] == 0).all()
    q = torch.randn(1, 4, d, generator=g)
    s = lref.scores(q[0], bd, bt[0], kv)
    for i, p in enumerate(bt[0].tolist()):
        k = kc[p, :, :13 - 5 * i].double()
        for j in range(kv):
            most = (q[0, 2 * j:2 * j + 2].double() @ k[j].T).amax()
            assert float(s[j, i]) >= float(most) - 1e-12


def test_reference_bounds_in_two_parts():
    g = torch.Generator().manual_seed(2)
    kc = torch.randn(4, 1, 5, 3, generator=g)
    bt = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    old = torch.full((4, 1, 2, 3), 7.0)
    once = lref.bounds(kc, old, bt, [0], [12])
    twice = lref.bounds(kc, lref.bounds(kc, old, bt, [0], [7]), bt, [7], [12])
    assert torch.equal(once, twice) and (once[3] == 7).all()
    assert torch.equal(once[1, 0, 1], kc[1, 0, :2].amax(0))


def test_reference_select_by_hand():
    # one channel: the score of a block is max(q lo, q hi)
    bd = torch.tensor([[-1.0, 2.0], [-5.0, 0.0], [0.0, 2.0], [1.0, 1.0]]).reshape(4, 1, 2, 1)
    bt = torch.tensor([[0, 1, 2, 3], [0, 1, 2, -1]], dtype=torch.int32)
    q = torch.tensor([[[1.0]], [[-1.0]]])
    lens = torch.tensor([40, 40])
    got = lref.select(q, bd, bt, lens, 10, 2, 0, 0)
    assert got.tolist() == [[[0, 2]], [[0, 1]]]  # scores 2 0 2 1 and 1 5 0
    assert lref.select(q, bd, bt, lens, 10, 3, 0, 1).tolist() == [[[0, 2, 3]], [[0, 1, 2]]]
    assert lref.select(q, bd, bt, torch.tensor([15, 0]), 10, 3, 1, 1).tolist() == [[[0, 1, -1]], [[-1, -1, -1]]]


def test_reference_attention_of_everything_is_the_paged_one():
    g = torch.Generator().manual_seed(3)
    page, kv, h, d = 5, 2, 6, 16
    k, v = (torch.randn(9, kv, page, d, generator=g) for _ in range(2))
    lens = torch.tensor([0, 1, 12], dtype=torch.int32)
    bt = torch.tensor([[-1, -1, -1], [4, -1, -1], [7, 0, 3]], dtype=torch.int32)
    q = torch.randn(3, h, d, generator=g)
    want, wlse, _, _ = ref.attention(q, k, v, bt, lens, 0.3)
    sel = torch.tensor([0, 1, 2], dtype=torch.int32).expand(3, kv, 3)
    out, lse, _, _ = lref.over(q, lref.Chosen((k, v), bt, lens, sel), 0.3)
    assert torch.allclose(out, want) and torch.allclose(lse, wlse)
    own = torch.tensor([0, 1, 2], dtype=torch.int32)
    out, lse, _, _ = lref.over(q, lref.Behind((k, v), bt[2], 12, bt[2:].expand(3, 3), own * 0), 0.3)
    one, _, _, _ = ref.attention(q, k, v, bt[2:].expand(3, 3), torch.tensor([12, 12, 12]), 0.3)
    assert torch.allclose(out, one)


# ------------------------------------------------------------ C refusals
SHAPE = dict(T=4, H=8, HK=2, d=64, dtype=la.LA_DTYPE_BF16)
CACHE = dict(kc=A, kps=2 * 16 * 64, vc=A + 0x80000, vps=2 * 16 * 64)
TABLE = dict(bt=A, bts=5, btw=5, lens=A, pages=10, page=16)

SHAPES = [(dict(T=-1), BAD), (dict(HK=0), BAD), (dict(d=96), BAD), (dict(dtype=5), BAD), (dict(T=0), la.LA_OK)]
TABLES = [(dict(bt=None), BAD), (dict(lens=None), BAD), (dict(lens=A + 2), BAD), (dict(bts=4), BAD),
          (dict(btw=-1), BAD), (dict(page=0), BAD), (dict(pages=-1), BAD), (dict(pages=2 ** 27), BAD)]
QUERIES = [(dict(q=None), BAD), (dict(q=A + 8), BAD), (dict(qs=511), BAD), (dict(qs=516), BAD), (dict(H=7), BAD),
           (dict(H=0), BAD)]
WORK = [(dict(ws=None), BAD), (dict(ws=A + 8), BAD), (dict(wsb=100), BAD)]
KEYS = [(dict(kc=None), BAD), (dict(kc=A + 4), BAD), (dict(kps=2047), BAD), (dict(kps=2052), BAD)]
VALUES = [(dict(vc=None), BAD), (dict(vps=2047), BAD)]
OUTPUTS = [(dict(out=None), BAD), (dict(out=A + 4), BAD), (dict(lse=A + 2), BAD), (dict(scale=float("nan")), BAD)]


def _bounds(lib, **kw):
    a = dict(bd=A + 0x40000, bps=2 * 2 * 64, first=A, **SHAPE, **CACHE, **TABLE)
    a.update(kw)
    return lib.lightning_attn_paged_bounds(a["kc"], a["kps"], a["bd"], a["bps"], a["bt"], a["bts"], a["btw"],
                                           a["first"], a["lens"], a["pages"], a["page"], a["T"], a["HK"],
                                           a["d"], a["dtype"], None)


@pytest.mark.parametrize("kw, status", SHAPES + TABLES + KEYS + [
    (dict(bd=None), BAD), (dict(bd=A + 0x40008), BAD), (dict(bps=255), BAD), (dict(bd=A), BAD),
    (dict(first=None), BAD), (dict(first=A + 1), BAD), (dict(pages=0), la.LA_OK)])
def test_paged_bounds_refusals(lib, kw, status):
    assert _bounds(lib, **kw) == status


def _select(lib, **kw):
    a = dict(q=A, qs=512, bd=A, bps=2 * 2 * 64, count=4, first=1, last=1, sel=A, ws=A, wsb=1 << 30, **SHAPE, **TABLE)
    a.update(kw)
    return lib.lightning_attn_paged_select(a["q"], a["qs"], a["bd"], a["bps"], a["bt"], a["bts"], a["btw"],
                                           a["lens"], a["pages"], a["page"], a["T"], a["H"], a["HK"], a["d"],
                                           a["dtype"], a["count"], a["first"], a["last"], a["sel"], a["ws"],
                                           a["wsb"], None)


@pytest.mark.parametrize("kw, status", SHAPES + TABLES + QUERIES + WORK + [
    (dict(bd=None), BAD), (dict(bps=252), BAD), (dict(count=0), BAD), (dict(first=-1), BAD), (dict(last=-1), BAD),
    (dict(first=3, last=2), BAD), (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), BAD), (dict(sel=None), BAD),
    (dict(sel=A + 2), BAD)])
def test_paged_select_refusals(lib, kw, status):
    assert _select(lib, **kw) == status


def _sparse(lib, **kw):
    a = dict(q=A, qs=512, sel=A, count=4, scale=0.1, out=A, lse=None, ws=A, wsb=1 << 30, **SHAPE, **CACHE, **TABLE)
    a.update(kw)
    return lib.lightning_attn_paged_sparse_decode(
        a["q"], a["qs"], a["kc"], a["kps"], a["vc"], a["vps"], a["bt"], a["bts"], a["btw"], a["lens"],
        a["sel"], a["count"], a["pages"], a["page"], a["T"], a["H"], a["HK"], a["d"], a["dtype"], a["scale"],
        a["out"], a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw, status", SHAPES + TABLES + QUERIES + WORK + KEYS + VALUES + OUTPUTS + [
    (dict(sel=None), BAD), (dict(sel=A + 2), BAD), (dict(count=0), BAD),
    (dict(count=2 ** 27), la.LA_ERR_UNSUPPORTED)])
def test_paged_sparse_decode_refusals(lib, kw, status):
    assert _sparse(lib, **kw) == status
    if status:
        assert lib.lightning_attn_last_error().decode() != ""


def _prefix(lib, **kw):
    a = dict(q=A, qs=512, pt=A, pw=7, pl=A, scale=0.1, out=A, lse=None, ws=A, wsb=1 << 30, **SHAPE, **CACHE, **TABLE)
    a.update(kw)
    return lib.lightning_attn_paged_prefix_decode(
        a["q"], a["qs"], a["kc"], a["kps"], a["vc"], a["vps"], a["pt"], a["pw"], a["pl"], a["bt"], a["bts"],
        a["btw"], a["lens"], a["pages"], a["page"], a["T"], a["H"], a["HK"], a["d"], a["dtype"], a["scale"],
        a["out"], a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw, status", SHAPES + TABLES + QUERIES + WORK + KEYS + VALUES + OUTPUTS + [
    (dict(pt=None), BAD), (dict(pt=A + 2), BAD), (dict(pl=None), BAD), (dict(pl=A + 1), BAD), (dict(pw=-1), BAD)])
def test_paged_prefix_decode_refusals(lib, kw, status):
    assert _prefix(lib, **kw) == status
    if status:
        assert lib.lightning_attn_last_error().decode() != ""


def test_prefix_workspace_sizes(lib):
    size = lib.lightning_attn_paged_prefix_decode_workspace_bytes
    for dtype in (0, 1):
        assert size(1, 8, 8, 128, dtype) > la.paged_decode_workspace_bytes(128)
        assert size(128, 64, 8, 128, dtype) > size(1, 64, 8, 128, dtype) and size(0, 1, 1, 64, dtype) > 0
    for bad in ((-1, 8, 8, 64, 0), (1, 0, 1, 64, 0), (1, 8, 0, 64, 0), (1, 8, 3, 64, 0), (1, 8, 8, 32, 0),
                (1, 8, 8, 64, 2), (2 ** 30, 8, 8, 64, 0)):
        assert size(*bad) == -1


def test_select_workspace_sizes(lib):
    size = lib.lightning_attn_paged_select_workspace_bytes
    assert size(1, 1, 100) >= 1200 and size(0, 1, 0) >= 0
    assert size(128, 8, 512) > 128 * 8 * 512 * 12
    assert size(-1, 1, 1) == -1 and size(1, 0, 1) == -1 and size(1, 1, -1) == -1
    assert size(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1) == -1


def test_binding_refuses_cpu_tensors():
    q, k = torch.zeros(2, 4, 64), torch.zeros(3, 2, 16, 64)
    i, bt = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    sel = torch.zeros(2, 2, 1, dtype=torch.int32)
    for call in (lambda: la.paged_bounds(k, k[:, :, :2], bt, i, i), lambda: la.paged_select(q, k[:, :, :2], bt, i, 16, 1),
                 lambda: la.paged_sparse_decode(q, k, k, bt, i, sel),
                 lambda: la.paged_prefix_decode(q, k, k, i, i[:1], bt, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
