"""Softmax-layer operators without a GPU: the reference checks itself (its
gradients against differences, its paged attention against a dense one), and
the library and binding refuse bad calls before anything is launched."""
import pytest
import torch

import softmax_reference as ref
import lightning_attention_attn_gb300 as la
from lightning_attention_attn_gb300 import build as labuild

A = 0x100000  # an aligned fake address: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    return la.load(labuild.build())


# --------------------------------------------------------------- reference
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32])
def test_reference_gradient_against_differences(interleaved, rot):
    g = torch.Generator().manual_seed(rot + interleaved)
    t, h, d, eps = 3, 2, 32, 1e-3
    x, dy = (torch.randn(t, h, d, generator=g, dtype=torch.float64) for _ in range(2))
    w = torch.randn(d, generator=g, dtype=torch.float64)
    table = la.rotary_table(50, rot, device="cpu") if rot else None
    pos = torch.tensor([0, 7, 49], dtype=torch.int32)

    def loss(x, w):
        return (ref.norm_rope(x, w, eps, table, pos, interleaved)[0] * dy).sum()

    dx, dw, _, _ = ref.norm_rope_backward(x, w, eps, table, pos, interleaved, dy)
    step = 1e-6
    for v, grad, at in ((x, dx, 0), (w, dw, 1)):
        way = torch.randn(v.shape, generator=g, dtype=torch.float64)
        args = [x, w]
        args[at] = v + step * way
        up = loss(*args)
        args[at] = v - step * way
        slope = (up - loss(*args)) / (2 * step)
        # central difference: step^2 truncation and 1e-16 / step rounding
        assert abs(float(slope - (grad * way).sum())) < 1e-7


def test_reference_attention_is_the_dense_one():
    g = torch.Generator().manual_seed(0)
    page, hk, h, d = 5, 2, 6, 64
    lens = torch.tensor([0, 1, 12], dtype=torch.int32)
    k, v = (torch.randn(9, hk, page, d, generator=g) for _ in range(2))
    bt = torch.tensor([[-1, -1, -1], [4, -1, -1], [7, 0, 3]], dtype=torch.int32)
    q = torch.randn(3, h, d, generator=g)
    out, lse, _, _ = ref.attention(q, k, v, bt, lens, 0.3)
    assert (out[0] == 0).all() and torch.isinf(lse[0]).all()
    kk = torch.cat([k[7], k[0], k[3]], dim=1)[:, :12].double()
    vv = torch.cat([v[7], v[0], v[3]], dim=1)[:, :12].double()
    for j in range(h):
        s = kk[j // 3] @ q[2, j].double() * 0.3
        assert torch.allclose(out[2, j], torch.softmax(s, 0) @ vv[j // 3])
        assert torch.allclose(lse[2, j], torch.logsumexp(s, 0))
        assert torch.allclose(out[1, j], v[4, j // 3, 0].double())


def test_reference_reserve_by_hand():
    r = ref.reserve([[5, -1], [1, 2], [-1, -1]], [3, 6, 0], [2, 1, 4], [False, True, False],
                    [0, 3, -1, -1, -1, -1], 2, 4, 9)
    # request 1 returns pages 1 and 2: stack 0 3 1 2; request 0 needs one (2), 1 one (1), 2 one (3)
    assert r["table"] == [[5, 2], [1, 2], [3, -1]] and r["count"] == 1
    assert r["slots"] == [5 * 4 + 3, 2 * 4, 1 * 4, 12, 13, 14, 15, -1, -1]
    assert r["lens"] == [5, 1, 4] and r["cu"] == [0, 2, 3, 7] and r["served"] == [True] * 3


def test_rotary_table():
    t = la.rotary_table(1 << 17, 64, base=10000.0)
    assert t.shape == (1 << 17, 64) and t.dtype == torch.float32
    p, i = 131071, 3
    angle = torch.tensor(p * 10000.0 ** (-2 * i / 64), dtype=torch.float64)
    assert abs(float(t[p, i]) - float(angle.cos())) <= ref.E
    assert abs(float(t[p, 32 + i]) - float(angle.sin())) <= ref.E
    for bad in (8, 24, 0):
        with pytest.raises(ValueError):
            la.rotary_table(4, bad)


# ------------------------------------------------------------ C refusals
ROTARY = dict(positions=A, rotary=A, rows=64, rot=64, interleaved=0, qw=A, kw=A, eps=1e-6)
SHAPE = dict(T=4, H=8, HK=2, d=64, dtype=la.LA_DTYPE_BF16)
CACHE = dict(kc=A, kps=2 * 16 * 64, vc=A + 0x80000, vps=2 * 16 * 64)


def _norm(lib, **kw):
    a = dict(q=A, qs=512, k=A, ks=128, qo=A + 0x1000, qos=512, ko=A + 0x2000, kos=128,
             **ROTARY, **SHAPE)
    a.update(kw)
    return lib.lightning_attn_qk_norm_rope(
        a["q"], a["qs"], a["k"], a["ks"], a["positions"], a["rotary"], a["rows"], a["rot"],
        a["interleaved"], a["qw"], a["kw"], a["eps"], a["T"], a["H"], a["HK"], a["d"], a["dtype"],
        a["qo"], a["qos"], a["ko"], a["kos"], None)


COMMON = [
    (dict(T=-1), la.LA_ERR_INVALID_ARG),
    (dict(H=0), la.LA_ERR_INVALID_ARG),
    (dict(HK=-1), la.LA_ERR_INVALID_ARG),
    (dict(d=96), la.LA_ERR_INVALID_ARG),
    (dict(dtype=5), la.LA_ERR_INVALID_ARG),
    (dict(q=None), la.LA_ERR_INVALID_ARG),
    (dict(q=A + 8), la.LA_ERR_INVALID_ARG),
    (dict(qs=511), la.LA_ERR_INVALID_ARG),
    (dict(qs=516), la.LA_ERR_INVALID_ARG),                 # 8 bytes past a 16-byte multiple
    (dict(ks=64), la.LA_ERR_INVALID_ARG),                  # rows overlap
    (dict(rot=8), la.LA_ERR_INVALID_ARG),
    (dict(rot=80), la.LA_ERR_INVALID_ARG),
    (dict(rows=0), la.LA_ERR_INVALID_ARG),
    (dict(rotary=None), la.LA_ERR_INVALID_ARG),
    (dict(positions=None), la.LA_ERR_INVALID_ARG),
    (dict(qw=None), la.LA_ERR_INVALID_ARG),                # one weight without the other
    (dict(eps=-1.0), la.LA_ERR_INVALID_ARG),
    (dict(eps=float("nan")), la.LA_ERR_INVALID_ARG),
    (dict(T=2 ** 30), la.LA_ERR_INVALID_ARG),              # too many rows
]


@pytest.mark.parametrize("kw, status", COMMON + [
    (dict(ko=None), la.LA_ERR_INVALID_ARG),
    (dict(qo=A, qos=640), la.LA_ERR_INVALID_ARG),          # in place with another stride
    (dict(HK=0), la.LA_ERR_INVALID_ARG),                   # a key weight without keys
    (dict(T=0), la.LA_OK),
])
def test_qk_norm_rope_refusals(lib, kw, status):
    assert _norm(lib, **kw) == status


def _back(lib, **kw):
    a = dict(q=A, qs=512, k=A + 0x800, ks=128, dqo=A + 0x1000, dqos=512, dko=A + 0x2000, dkos=128,
             dq=A + 0x3000, dqs=512, dk=A + 0x4000, dks=128, dqw=A, dkw=A, ws=A, wsb=1 << 30,
             **ROTARY, **SHAPE)
    a.update(kw)
    return lib.lightning_attn_qk_norm_rope_backward(
        a["q"], a["qs"], a["k"], a["ks"], a["positions"], a["rotary"], a["rows"], a["rot"],
        a["interleaved"], a["qw"], a["kw"], a["eps"], a["T"], a["H"], a["HK"], a["d"], a["dtype"],
        a["dqo"], a["dqos"], a["dko"], a["dkos"], a["dq"], a["dqs"], a["dk"], a["dks"], a["dqw"],
        a["dkw"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw, status", COMMON + [
    (dict(dqw=None), la.LA_ERR_INVALID_ARG),
    (dict(dkw=None), la.LA_ERR_INVALID_ARG),
    (dict(ws=None), la.LA_ERR_INVALID_ARG),
    (dict(ws=A + 4), la.LA_ERR_INVALID_ARG),
    (dict(wsb=100), la.LA_ERR_INVALID_ARG),
    (dict(dq=A), la.LA_ERR_INVALID_ARG),                   # over an input that is still read
    (dict(dk=A + 0x3000), la.LA_ERR_INVALID_ARG),          # two gradients in one array
    (dict(dqo=None), la.LA_ERR_INVALID_ARG),
    (dict(qw=None, kw=None, T=0), la.LA_OK),
])
def test_qk_norm_rope_backward_refusals(lib, kw, status):
    assert _back(lib, **kw) == status


def _append(lib, **kw):
    a = dict(q=A, qs=512, k=A, ks=128, v=A, vs=128, qo=A + 0x1000, qos=512, slots=A, pages=10,
             page=16, **ROTARY, **SHAPE, **CACHE)
    a.update(kw)
    return lib.lightning_attn_paged_append(
        a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["positions"], a["rotary"], a["rows"],
        a["rot"], a["interleaved"], a["qw"], a["kw"], a["eps"], a["T"], a["H"], a["HK"], a["d"],
        a["dtype"], a["qo"], a["qos"], a["kc"], a["kps"], a["vc"], a["vps"], a["slots"], a["pages"],
        a["page"], None)


POOL = [
    (dict(HK=0), la.LA_ERR_INVALID_ARG),
    (dict(kc=None), la.LA_ERR_INVALID_ARG),
    (dict(vc=A + 4), la.LA_ERR_INVALID_ARG),
    (dict(kps=2047), la.LA_ERR_INVALID_ARG),
    (dict(vps=2052), la.LA_ERR_INVALID_ARG),
    (dict(page=0), la.LA_ERR_INVALID_ARG),
    (dict(pages=-1), la.LA_ERR_INVALID_ARG),
    (dict(pages=2 ** 27), la.LA_ERR_INVALID_ARG),          # slots pass 32 bits
]


@pytest.mark.parametrize("kw, status", COMMON + POOL + [
    (dict(v=None), la.LA_ERR_INVALID_ARG),
    (dict(slots=None), la.LA_ERR_INVALID_ARG),
    (dict(slots=A + 2), la.LA_ERR_INVALID_ARG),
    (dict(T=0), la.LA_OK),
])
def test_paged_append_refusals(lib, kw, status):
    assert _append(lib, **kw) == status
    if status:
        assert lib.lightning_attn_last_error().decode() != ""


def _decode(lib, **kw):
    a = dict(q=A, qs=512, bt=A, bts=5, btw=5, lens=A, pages=10, page=16, scale=0.1, out=A + 0x1000,
             lse=None, ws=A, wsb=1 << 30, **SHAPE, **CACHE)
    a.update(kw)
    return lib.lightning_attn_paged_decode(
        a["q"], a["qs"], a["kc"], a["kps"], a["vc"], a["vps"], a["bt"], a["bts"], a["btw"],
        a["lens"], a["pages"], a["page"], a["T"], a["H"], a["HK"], a["d"], a["dtype"], a["scale"],
        a["out"], a["lse"], a["ws"], a["wsb"], None)


DECODE = [
    (dict(H=7), la.LA_ERR_INVALID_ARG),                    # not a multiple of the kv heads
    (dict(bt=None), la.LA_ERR_INVALID_ARG),
    (dict(lens=None), la.LA_ERR_INVALID_ARG),
    (dict(lens=A + 2), la.LA_ERR_INVALID_ARG),
    (dict(bts=4), la.LA_ERR_INVALID_ARG),
    (dict(btw=-1), la.LA_ERR_INVALID_ARG),
    (dict(scale=float("inf")), la.LA_ERR_INVALID_ARG),
    (dict(out=None), la.LA_ERR_INVALID_ARG),
    (dict(out=A + 4), la.LA_ERR_INVALID_ARG),
    (dict(lse=A + 2), la.LA_ERR_INVALID_ARG),
    (dict(ws=None), la.LA_ERR_INVALID_ARG),
    (dict(wsb=1000), la.LA_ERR_INVALID_ARG),
    (dict(T=0), la.LA_OK),
]


@pytest.mark.parametrize("kw, status", [c for c in COMMON if not set(c[0]) & (set(ROTARY) | {"ks"})] +
                         POOL + DECODE)
def test_paged_decode_refusals(lib, kw, status):
    assert _decode(lib, **kw) == status


def _step(lib, **kw):
    a = dict(q=A, qs=512, k=A, ks=128, v=A, vs=128, slots=A, bt=A, bts=5, btw=5, lens=A, pages=10,
             page=16, scale=0.1, out=A + 0x1000, lse=None, ws=A, wsb=1 << 30, **ROTARY, **SHAPE, **CACHE)
    a.update(kw)
    return lib.lightning_attn_paged_step(
        a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["positions"], a["rotary"], a["rows"],
        a["rot"], a["interleaved"], a["qw"], a["kw"], a["eps"], a["kc"], a["kps"], a["vc"],
        a["vps"], a["slots"], a["bt"], a["bts"], a["btw"], a["lens"], a["pages"], a["page"],
        a["T"], a["H"], a["HK"], a["d"], a["dtype"], a["scale"], a["out"], a["lse"], a["ws"],
        a["wsb"], None)


@pytest.mark.parametrize("kw, status", COMMON + POOL + DECODE +
                         [(dict(slots=None), la.LA_ERR_INVALID_ARG)])
def test_paged_step_refusals(lib, kw, status):
    assert _step(lib, **kw) == status


def _reserve(lib, **kw):
    a = dict(bt=A, bts=5, btw=5, lens=A, new=A, done=None, B=4, stack=A, count=A, pages=10, page=16,
             T=4, slots=A, pos=A, cu=A, served=A, lo=A, co=A)
    a.update(kw)
    return lib.lightning_attn_paged_reserve(
        a["bt"], a["bts"], a["btw"], a["lens"], a["new"], a["done"], a["B"], a["stack"], a["count"],
        a["pages"], a["page"], a["T"], a["slots"], a["pos"], a["cu"], a["served"], a["lo"], a["co"],
        None)


@pytest.mark.parametrize("kw, status", [
    (dict(B=0), la.LA_ERR_INVALID_ARG),
    (dict(B=8193), la.LA_ERR_UNSUPPORTED),
    (dict(T=-1), la.LA_ERR_INVALID_ARG),
    (dict(page=0), la.LA_ERR_INVALID_ARG),
    (dict(pages=2 ** 30), la.LA_ERR_INVALID_ARG),
    (dict(bts=4), la.LA_ERR_INVALID_ARG),
    (dict(new=None), la.LA_ERR_INVALID_ARG),
    (dict(stack=None), la.LA_ERR_INVALID_ARG),
    (dict(slots=None), la.LA_ERR_INVALID_ARG),
    (dict(served=None), la.LA_ERR_INVALID_ARG),
    (dict(cu=A + 2), la.LA_ERR_INVALID_ARG),
])
def test_paged_reserve_refusals(lib, kw, status):
    assert _reserve(lib, **kw) == status


def test_workspace_sizes(lib):
    assert la.paged_decode_workspace_bytes(128) > 0
    assert la.paged_step_workspace_bytes(3, 8, 64) - la.paged_decode_workspace_bytes(64) == \
        3 * 8 * 64 * 4
    assert lib.lightning_attn_paged_decode_workspace_bytes(96) == -1
    assert lib.lightning_attn_paged_step_workspace_bytes(-1, 8, 64) == -1
    assert lib.lightning_attn_qk_norm_rope_workspace_bytes(32) == -1
    with pytest.raises(ValueError):
        la.paged_decode_workspace_bytes(100)


def test_binding_refuses_cpu_tensors():
    q, c = torch.zeros(2, 4, 64), torch.zeros(3, 2, 16, 64)
    i = torch.zeros(2, dtype=torch.int32)
    bt = torch.zeros(2, 3, dtype=torch.int32)
    for call in (lambda: la.qk_norm_rope(q, None),
                 lambda: la.qk_norm_rope_backward(q, None, None, None, q, None),
                 lambda: la.paged_append(q, q, q, i, None, c, c, i),
                 lambda: la.paged_decode(q, c, c, bt, i),
                 lambda: la.paged_step(q, q, q, i, None, c, c, i, bt, i),
                 lambda: la.paged_reserve(bt, i, i, i, i[:1], 16, 2)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
