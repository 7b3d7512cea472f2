"""GPU parity of the softmax layers' operators for long contexts (page bounds, choice of pages,
attention over chosen pages) against the 64-bit reference, at the sizes and masks where they can
go wrong, and a serving loop of them together."""
import math

import pytest
import torch

import long_context_reference as lref
import softmax_reference as ref
import lightning_attention_attn_gb300 as la
from lightning_attention_attn_gb300 import build as labuild

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.load(labuild.build())
    yield
    torch.cuda.synchronize()
    la.device_status()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def c(x):
    return None if x is None else x.cpu()


def tables(blocks, g, spare=2, extra=1):
    """Rows of a table with pages in random places; returns it and the pool's size."""
    pages = sum(blocks) + spare
    order = torch.randperm(pages, generator=g, device="cuda").int()
    bt = torch.full((len(blocks), max(max(blocks), 1) + extra), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(blocks):
        bt[b, :n] = order[at:at + n]
        at += n
    return bt, pages


def blocks_of(lens, page):
    return [-(-n // page) for n in lens]


# ------------------------------------------------------------------ bounds
def same(a, b):
    a, b = a.cpu().float(), b.float()
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert torch.equal(a[~torch.isnan(a)], b[~torch.isnan(b)])


@pytest.mark.parametrize("dtype, hk, d", [(BF16, 8, 128), (BF16, 3, 64), (FP32, 2, 128), (FP32, 1, 64)])
@pytest.mark.parametrize("page", [1, 5, 16, 64, 200])
def test_bounds(dtype, hk, d, page):
    g = gen(page + d)
    first = [0, 0, 7, 63, 64, 65, 129, 300, 40, 0, 11]
    lens = [1, 0, 7, 64, 65, 200, 131, 900, 20, 515, 12]  # the third and the ninth have nothing new
    bt, pages = tables(blocks_of(lens, page), g)
    kc, old = randn((pages, hk, page, d), dtype, g), randn((pages, hk, 2, d), dtype, g)
    got = old.clone()
    out = la.paged_bounds(kc, got, bt, ints(first), ints(lens))
    assert out.data_ptr() == got.data_ptr()
    same(got, lref.bounds(c(kc), c(old), c(bt), first, lens))
    again = old.clone()  # the same call gives the same bits
    assert torch.equal(la.paged_bounds(kc, again, bt, ints(first), ints(lens)), got)


def test_bounds_special_values_absent_pages_and_strides():
    g = gen(3)
    page, hk, d = 16, 2, 64
    lens = [70, 33, 5]
    bt, pages = tables(blocks_of(lens, page), g)
    both = randn((pages, 3, hk, page, d), BF16, g)  # pages of a wider array
    kc = both[:, 1]
    kc[bt[0, 0].long(), 0, 3, 5] = NAN
    kc[bt[0, 1].long(), 1, 0, 6], kc[bt[0, 1].long(), 1, 1, 6] = INF, -INF
    kc[bt[1, 2].long(), 0, 0, 1] = INF
    kc[bt[1, 2].long(), 0, 1:] = NAN  # behind the last token
    wide = torch.full((pages, 2 * hk, 2, d), 9.0, dtype=BF16, device="cuda")
    got = wide[:, :hk]
    bt[0, 2] = -1
    bt[2, 0] = 10 ** 9
    first, n = ints([-5, 0, 0]), ints([70, 33, 2 ** 31 - 1])
    la.paged_bounds(kc, got, bt, first, n)
    want = lref.bounds(c(kc), torch.full((pages, hk, 2, d), 9.0, dtype=BF16), c(bt), c(first), c(n))
    same(got, want)
    assert (wide[:, hk:] == 9).all()
    assert torch.isnan(got[bt[0, 0].long(), 0, :, 5]).all()


def test_bounds_refusals():
    g = gen(4)
    kc, bd = randn((4, 2, 16, 64), BF16, g), randn((4, 2, 2, 64), BF16, g)
    bt, n = torch.zeros((3, 4), dtype=torch.int32, device="cuda"), ints([1, 2, 3])
    before = bd.clone()
    for bad in (dict(bd=bd.float()), dict(bd=bd[:3]), dict(bd=bd[:, :1]), dict(bd=kc), dict(bt=bt.long()),
                dict(first=n[:2]), dict(lens=n.long()), dict(kc=kc.transpose(1, 2)), dict(bt=bt[0]),
                dict(bd=bd.cpu()), dict(kc=kc[0])):
        a = {**dict(kc=kc, bd=bd, bt=bt, first=n, lens=n), **bad}
        with pytest.raises((ValueError, la.LightningAttnError)):
            la.paged_bounds(a["kc"], a["bd"], a["bt"], a["first"], a["lens"])
    with pytest.raises(TypeError):
        la.paged_bounds(kc.half(), bd.half(), bt, n, n)
    la.paged_bounds(kc, bd, bt[:0], n[:0], n[:0])
    assert torch.equal(bd, before)


# ------------------------------------------------------------------ choice
def some_bounds(pages, hk, d, dtype, g):
    mid = torch.randn((pages, hk, d), generator=g, device="cuda")
    reach = 0.5 + 2 * torch.rand((pages, hk, d), generator=g, device="cuda")
    return torch.stack([mid * 0.5 - reach, mid * 0.5 + reach], 2).to(dtype)


def check_select(q, bd, bt, lens, page, count, first=1, last=1):
    out = la.paged_select(q, bd, bt, lens, page, count, keep_first=first, keep_last=last)
    want = lref.select(c(q), c(bd), c(bt), c(lens), page, count, first, last)
    assert torch.equal(out.cpu(), want)
    return out


SELECT_LENS = [0, 1, 16, 17, 100, 256, 257, 512, 513, 4000, 15000, 1, 0]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d, h, hk", [(128, 64, 8), (64, 3, 3), (128, 7, 1), (64, 18, 2), (128, 33, 1)])
def test_select(dtype, d, h, hk):
    g = gen(d + h)
    page = 16
    bt, pages = tables(blocks_of(SELECT_LENS, page), g)
    bd = some_bounds(pages, hk, d, dtype, g)
    q = randn((len(SELECT_LENS), h, d), dtype, g)
    for count, first, last in ((1, 0, 0), (1, 1, 0), (2, 1, 1), (17, 0, 3), (64, 4, 2), (250, 1, 1), (1000, 0, 0)):
        check_select(q, bd, bt, ints(SELECT_LENS), page, count, first, last)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_select_near_and_equal_scores(dtype):
    """Blocks whose scores are equal, or differ by less than fp32 sums resolve: the order is that of
    64-bit scores, ties to the lower block; more of them than are ranked one against the other, too."""
    g = gen(7)
    d, page, n = 128, 16, 400
    bt, pages = tables([n] * 3, g)
    base = some_bounds(1, 1, d, dtype, g)
    bd = base.expand(pages, 1, 2, d).clone()  # request 0: all blocks equal
    # request 1: one channel in 100 of them differs by the type's last bit, in either direction
    # (its contribution is small against the sum), others are copies of those
    eps = torch.finfo(dtype).eps
    step = (torch.randint(-3, 4, (100,), generator=g, device="cuda").float() * eps * 0.25)
    small = bd[bt[1, 50:150].long(), 0, 1, 7].float() * 2.0 ** -8
    bd[bt[1, :n].long(), 0, :, 7] = 0
    bd[bt[1, 50:150].long(), 0, 1, 7] = (small * (1 + 4 * step)).to(dtype)
    # request 2: a few blocks above the others, the border inside a run of equal ones
    bd[bt[2, 10:20].long(), 0, 1] *= 2
    q = randn((3, 8, d), dtype, g)
    q[1, :, 7] = q[1, :, 7].abs()
    for count in (1, 5, 30, 64, 65, 120, 399):
        check_select(q, bd, bt, ints([n * page, n * page - 3, n * page]), page, count, 0, 1)


def test_select_cancelling_sums():
    """Scores of a few units from terms of thousands: fp32 sums are off by more than the scores
    differ, in any order; the choice is that of the true ones."""
    g = gen(8)
    d, page, n = 64, 8, 700
    bt, pages = tables([n, n], g)
    for dtype in (BF16, FP32):
        x = (torch.randn((pages, 2, 1, d), generator=g, device="cuda") * 4000).to(dtype)
        x[..., 32:] = x[..., :32]  # q's second half is the first one's negative
        x = x.expand(pages, 2, 2, d).clone()
        tail = torch.randn((pages, 2, 2, 1), generator=g, device="cuda") * 2 ** -6
        x[..., 63:] = x[..., 63:] * 0 + tail.to(dtype)
        x[..., 31] = 0
        q = randn((2, 4, d), dtype, g)
        q[..., 32:63] = -q[..., :31]
        check_select(q, x.contiguous(), bt, ints([n * page, n * page]), page, 40, 0, 0)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("of_q, of_k", [(-70, -72), (-60, -60), (-74, -74), (0, -131), (-131, 0), (60, -138)])
def test_select_tiny_numbers(dtype, of_q, of_k):
    """Scores (or queries, or bounds) in and below the subnormal range of fp32, where an error is not
    relative to its terms: exact in 64 bits, and so is the choice."""
    g = gen(9)
    page, n = 16, 300
    bt, pages = tables([n] * 4, g)
    bd = (some_bounds(pages, 2, 64, FP32, g).double() * 2.0 ** of_k).to(dtype)
    q = (torch.randn((4, 6, 64), generator=g, device="cuda").double() * 2.0 ** of_q).to(dtype)
    for count in (1, 20, 100):
        check_select(q, bd, bt, ints([n * page] * 4), page, count, 0, 0)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_select_infinities_nan_and_absent_pages(dtype):
    g = gen(9)
    d, page, n = 64, 16, 200
    bt, pages = tables([n] * 4, g)
    bd = some_bounds(pages, 2, d, dtype, g)
    q = randn((4, 8, d), dtype, g)
    bd[bt[0, 5].long(), 0, 0, 3], bd[bt[0, 9].long(), 0, 1, 3] = NAN, INF
    bd[bt[0, 11].long(), 1, :, 4] = -INF  # infinite for one sign of q, minus infinity for the other
    bd[bt[1, 20].long(), 1, 0, 0] = -INF
    q[2, 1, 5] = INF
    q[3, 6] = 0  # a head of zeros beside others
    bt[0, 30:60] = -1                      # no pages: never chosen, not even the first and the last
    bt[1, 0], bt[1, n - 1] = 10 ** 9, -3
    check_select(q, bd, bt, ints([n * page] * 4), page, 20, 2, 2)
    bt[2, 10:] = -1                        # fewer pages than are asked for
    check_select(q, bd, bt, ints([n * page, -4, n * page, 2 ** 31 - 1]), page, 20, 2, 2)
    # what other requests' pages hold does not matter
    bd[bt[3, :n].long()] = NAN
    check_select(q[:2], bd, bt[:2], ints([n * page] * 2), page, 64)


def test_select_strides_refusals_and_own_output():
    g = gen(10)
    d, page, n, hk = 64, 16, 90, 2
    bt, pages = tables([n, n, 3], g)
    wide = randn((pages, 3 * hk, 2, d), BF16, g).abs()
    bd = wide[:, hk:2 * hk]
    bd[:, :, 0] = -bd[:, :, 0]
    x = randn((3, 10, d), BF16, g)
    lens = ints([n * page, 900, 40])
    want = check_select(x[:, 2:8], bd, bt, lens, page, 9)
    out = torch.full((5, hk, 9), 7, dtype=torch.int32, device="cuda")
    ws = torch.empty(la.paged_select_workspace_bytes(3, hk, bt.shape[1]), dtype=torch.uint8, device="cuda")
    got = la.paged_select(x[:, 2:8], bd, bt, lens, page, 9, out=out[1:4], workspace=ws)
    assert torch.equal(got, want) and (out[0] == 7).all() and (out[4] == 7).all()
    q = x[:, 2:8]
    for kw in (dict(count=0), dict(count=2, keep_first=2), dict(keep_last=-1), dict(page=0), dict(out=out[:2]),
               dict(q=x[:, :7]), dict(lens=lens.long()), dict(ws=ws[:-16]), dict(bd=bd[:, :, :1]),
               dict(bd=bd.float())):
        a = {**dict(count=9, keep_first=1, keep_last=1, page=page, out=None, q=q, lens=lens, ws=None, bd=bd), **kw}
        with pytest.raises((ValueError, la.LightningAttnError)):
            la.paged_select(a["q"], a["bd"], bt, a["lens"], a["page"], a["count"], keep_first=a["keep_first"],
                            keep_last=a["keep_last"], out=a["out"], workspace=a["ws"])
    assert la.paged_select(q[:0], bd, bt[:0], lens[:0], page, 4).shape == (0, hk, 4)


# -------------------------------------------------- attention over chosen pages
def caches(pages, hk, page, d, dtype, g):
    return tuple(randn((pages, hk, page, d), dtype, g) for _ in range(2))


def some_choice(lens, page, hk, count, g, sort=True):
    sel = torch.full((len(lens), hk, count), -1, dtype=torch.int32)
    cpu = torch.Generator().manual_seed(count)
    for b, n in enumerate(lens):
        blocks = -(-n // page)
        for j in range(hk):
            got = torch.randperm(blocks, generator=cpu)[:count]
            if len(got) and blocks - 1 not in got:
                got[0] = blocks - 1
            sel[b, j, :len(got)] = (got.sort().values if sort else got).int()
    return sel.cuda()


def check_sparse(q, kc, vc, bt, lens, sel, scale=None, **kw):
    b, h, d = q.shape
    lse = torch.empty((b, h), device="cuda")
    out = la.paged_sparse_decode(q, kc, vc, bt, lens, sel, scale=scale, lse=lse, **kw)
    scale = d ** -0.5 if scale is None else scale
    want, wlse, bound, lbound = lref.over(c(q), lref.Chosen((c(kc), c(vc)), c(bt), c(lens), c(sel)), scale)
    ref.within(out, want, bound, ref.u_of(q.dtype), "out")
    ref.within(lse, wlse, lbound, ref.u_of(FP32), "lse")
    return out


SPARSE_LENS = [0, 1, 16, 17, 100, 256, 257, 512, 513, 2000, 5000, 1, 0]


@pytest.mark.parametrize("dtype, h, hk, d", [(BF16, 16, 2, 128), (BF16, 12, 1, 64), (FP32, 6, 2, 64),
                                             (FP32, 16, 1, 128), (BF16, 40, 2, 128)])
@pytest.mark.parametrize("page, count", [(1, 30), (5, 7), (16, 1), (16, 40), (64, 9), (200, 3)])
def test_sparse(dtype, h, hk, d, page, count):
    g = gen(page + count)
    bt, pages = tables(blocks_of(SPARSE_LENS, page), g)
    kc, vc = caches(pages, hk, page, d, dtype, g)
    sel = some_choice(SPARSE_LENS, page, hk, count, g, sort=page != 16)
    check_sparse(randn((len(SPARSE_LENS), h, d), dtype, g), kc, vc, bt, ints(SPARSE_LENS), sel)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_sparse_many_pages(dtype):
    """Enough chosen tokens for the split over all CTAs, ragged, and idle requests between."""
    g = gen(21)
    lens = [9000, 0, 3, 0, 20000, 700]
    page, hk, count = 32, 2, 300
    bt, pages = tables(blocks_of(lens, page), g)
    kc, vc = caches(pages, hk, page, 64, dtype, g)
    check_sparse(randn((6, 8, 64), dtype, g), kc, vc, bt, ints(lens), some_choice(lens, page, hk, count, g))


def test_sparse_of_all_pages_is_the_dense_one():
    g = gen(22)
    lens, page = [333, 64, 1, 2000], 16
    bt, pages = tables(blocks_of(lens, page), g)
    kc, vc = caches(pages, 2, page, 128, BF16, g)
    q = randn((4, 16, 128), BF16, g)
    sel = some_choice(lens, page, 2, 125, g)
    out = check_sparse(q, kc, vc, bt, ints(lens), sel)
    dense = la.paged_decode(q, kc, vc, bt, ints(lens))
    # one bf16 rounding of either, beside the two bounds' arithmetic (2^-16 and less)
    assert ((out.float() - dense.float()).abs() <= 2 ** -7 * dense.float().abs() + 1e-3).all()


def test_sparse_entries_that_are_none():
    """Entries outside the request's blocks, absent pages, a block twice, garbage behind the last
    token and in pages that are not chosen; a choice that holds nothing."""
    g = gen(23)
    lens, page, hk, d = [100, 40, 64, 9, 70], 16, 2, 128
    bt, pages = tables(blocks_of(lens, page), g)
    kc, vc = caches(pages, hk, page, d, BF16, g)
    sel = torch.full((5, hk, 6), -1, dtype=torch.int32, device="cuda")
    sel[0, 0] = ints([6, 2, 2, 10 ** 9, -7, 0])     # the last block (4 tokens), one twice, none
    sel[0, 1] = ints([7, 3, 5, 1, 6, 4])            # block 7 is not the request's
    sel[1, 0, :3] = ints([0, 1, 2])
    sel[1, 1, 3] = 0                                # past its three blocks: does not count
    sel[2, :, :4] = ints([1, 2, 3, 0])
    sel[3, 0, 0] = 0
    bt[2, 2], bt[2, 3] = -1, 10 ** 9
    sel[4, :, :5] = ints([2, 4, 2 ** 31 - 1, -2 ** 31, 0])
    for cache in (kc, vc):
        cache[bt[0, 6].long(), :, 4:] = NAN
        cache[bt[1, 2].long(), :, 8:] = NAN
        cache[bt[3, 0].long(), :, 9:] = NAN
        cache[bt[4, 4].long(), :, 6:] = NAN
        cache[bt[4, 1].long()] = cache[bt[4, 3].long()] = NAN
    out = check_sparse(randn((5, 8, d), BF16, g), kc, vc, bt, ints(lens), sel)
    assert (out[1, 4:] == 0).all() and (out[3, 4:] == 0).all()


def test_sparse_infinities_that_are_attended_to():
    g = gen(24)
    lens, page = [90, 90], 16
    bt, pages = tables(blocks_of(lens, page), g)
    kc, vc = caches(pages, 1, page, 128, BF16, g)
    sel = ints([[[0, 2, 5, -1, -1, -1]], [[1, 2, 3, -1, -1, -1]]])
    vc[bt[0, 2].long(), 0, 3, 7] = INF
    kc[bt[1, 2].long(), 0, 3] = INF   # the score's sum meets infinities of both signs
    vc[bt[0, 1].long()] = NAN         # not chosen
    q = randn((2, 4, 128), BF16, g)
    out = la.paged_sparse_decode(q, kc, vc, bt, ints(lens), sel)
    assert torch.isnan(out[1]).all() and (out[0, :, 7] == INF).all()
    assert torch.isfinite(out[0, :, :7]).all() and torch.isfinite(out[0, :, 8:]).all()


def test_sparse_refusals():
    g = gen(25)
    bt, pages = tables([3, 3], g)
    kc, vc = caches(pages, 2, 16, 64, BF16, g)
    q, lens = randn((2, 4, 64), BF16, g), ints([40, 40])
    sel = some_choice([40, 40], 16, 2, 2, g)
    for bad in (sel.long(), sel[:1], sel[:, :1], sel[:, :, :0], sel.transpose(0, 1), sel[..., ::2], sel.cpu()):
        with pytest.raises((ValueError, la.LightningAttnError)):
            la.paged_sparse_decode(q, kc, vc, bt, lens, bad)
    assert la.paged_sparse_decode(q[:0], kc, vc, bt[:0], lens[:0], sel[:0]).shape == (0, 4, 64)


# ------------------------------------------------------ behind a shared prefix
def behind(prefix, lens, page, hk, d, dtype, g, garbage=NAN):
    """A pool with the prefix and the requests' own tokens anywhere in it, garbage elsewhere."""
    bt, pages = tables(blocks_of([prefix] + lens, page), g)
    kc = torch.full((pages, hk, page, d), garbage, dtype=dtype, device="cuda")
    vc = kc.clone()
    for row, n in zip(bt, [prefix] + lens):
        t = torch.arange(n, device="cuda")
        for cache in (kc, vc):
            cache[row[t // page].long(), :, t % page] = randn((n, hk, d), dtype, g)
    return kc, vc, bt[0].clone(), ints([prefix]), bt[1:].clone(), ints(lens)


def check_prefix(q, kc, vc, pt, pl, bt, lens, scale=None, **kw):
    b, h, d = q.shape
    lse = torch.empty((b, h), device="cuda")
    out = la.paged_prefix_decode(q, kc, vc, pt, pl, bt, lens, scale=scale, lse=lse, **kw)
    scale = d ** -0.5 if scale is None else scale
    parts = lref.Behind((c(kc), c(vc)), c(pt), c(pl), c(bt), c(lens))
    want, wlse, bound, lbound = lref.over(c(q), parts, scale, tile=128)
    ref.within(out, want, bound, ref.u_of(q.dtype), "out")
    ref.within(lse, wlse, lbound, ref.u_of(FP32), "lse")
    return out


@pytest.mark.parametrize("dtype, h, hk, d", [(BF16, 16, 2, 128), (BF16, 12, 1, 64), (FP32, 6, 2, 64),
                                             (FP32, 16, 1, 128), (BF16, 40, 2, 128), (BF16, 3, 3, 64)])
@pytest.mark.parametrize("prefix, page", [(0, 16), (1, 16), (127, 1), (128, 64), (129, 48), (1000, 5), (4001, 64)])
def test_prefix(dtype, h, hk, d, prefix, page):
    g = gen(prefix + h)
    lens = [0, 1, 64, 65, 300]
    args = behind(prefix, lens, page, hk, d, dtype, g)
    out = check_prefix(randn((5, h, d), dtype, g), *args)
    if prefix == 0:
        assert (out[0] == 0).all()


@pytest.mark.parametrize("dtype, h, hk, d, batch", [
    (BF16, 8, 8, 128, 1), (BF16, 8, 8, 64, 3), (BF16, 64, 8, 128, 15), (BF16, 64, 8, 128, 16),
    (BF16, 64, 8, 128, 17), (BF16, 16, 1, 64, 16), (BF16, 7, 1, 128, 37), (BF16, 32, 2, 128, 41),
    (FP32, 4, 4, 64, 1), (FP32, 4, 1, 128, 2), (FP32, 16, 2, 64, 33), (BF16, 48, 1, 64, 11)])
def test_prefix_batches(dtype, h, hk, d, batch):
    """Rows of a key-value head from one to several hundred, in every relation to the tiles."""
    g = gen(batch + h)
    lens = [(37 * i) % 90 for i in range(batch)]
    args = behind(700, lens, 32, hk, d, dtype, g)
    check_prefix(randn((batch, h, d), dtype, g), *args)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [4, 8, 24, 128, 200, 256])
def test_prefix_page_sizes(page, d):
    """Pages that a tile's copies take as boxes of 8 to 128 rows, or row by row; absent pages of each."""
    g = gen(page)
    kc, vc, pt, pl, bt, sl = behind(1500, [30, 0, 7] * 7, page, 2, d, BF16, g)
    q = randn((21, 8, d), BF16, g)
    check_prefix(q, kc, vc, pt, pl, bt, sl)
    for gone in (1, 2, pt.numel() // 2, pt.numel() - 1):
        if gone < pt.numel():
            pt[gone] = -1 if gone % 2 else 2 ** 31 - 1
    check_prefix(q, kc, vc, pt, pl, bt, sl)
    check_prefix(q[:5], kc, vc, pt, pl, bt[:5], sl[:5])


@pytest.mark.parametrize("h, hk, batch, prefix", [(8, 8, 1, 5120), (16, 2, 4, 20000), (24, 12, 70, 2900),
                                                  (160, 160, 2, 100), (200, 200, 130, 300)])
@pytest.mark.parametrize("d", [64, 128])
def test_prefix_parts_of_several_units(h, hk, batch, prefix, d):
    """CTAs whose range ends one unit and begins another, or holds several units, with odd and even
    numbers of tiles of each."""
    g = gen(h + d)
    args = behind(prefix, [i % 3 for i in range(batch)], 64, hk, d, BF16, g, garbage=0.0)
    q = randn((batch, h, d), BF16, g)
    some = list(range(0, batch, 40))  # the reference for a few requests
    kc, vc, pt, pl, bt, sl = args
    out = la.paged_prefix_decode(q, *args)
    parts = lref.Behind((c(kc), c(vc)), c(pt), c(pl), c(bt[some]), c(sl[some]))
    want, _, bound, _ = lref.over(c(q[some]), parts, d ** -0.5, tile=128)
    ref.within(out[some], want, bound, ref.u_of(BF16), "out")
    la.device_status()


@pytest.mark.parametrize("h, hk, d", [(16, 2, 128), (12, 1, 64), (40, 1, 128), (8, 4, 64)])
@pytest.mark.parametrize("prefix", [100, 3000, 30000])
def test_prefix_beside_ragged_own_tokens(prefix, h, hk, d):
    """Few and many SMs for the prefix beside own tokens of every length, in one call after another
    over one workspace: whole requests, requests in many pieces, and none."""
    g = gen(prefix + h)
    lens = [(997 * i) % 600 if i % 5 else 0 for i in range(60)]
    lens[7], lens[31] = 9000, 5000
    kc, vc, pt, pl, bt, sl = behind(prefix, lens, 64, hk, d, BF16, g)
    q = randn((60, h, d), BF16, g)
    ws = torch.empty(la.paged_prefix_decode_workspace_bytes(60, h, hk, d), dtype=torch.uint8, device="cuda")
    some = [0, 1, 7, 13, 31, 59]
    for own in (sl, sl // 50, sl):  # (the second time the prefix gets nearly all SMs)
        out = la.paged_prefix_decode(q, kc, vc, pt, pl, bt, own, workspace=ws)
        parts = lref.Behind((c(kc), c(vc)), c(pt), c(pl), c(bt[some]), c(own[some]))
        want, _, bound, _ = lref.over(c(q[some]), parts, d ** -0.5, tile=128)
        ref.within(out[some], want, bound, ref.u_of(BF16), "out")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_prefix_long_and_wide(dtype):
    """A prefix of many tiles a CTA, own tokens for the split over all CTAs, a table much wider
    than the prefix, and the other way round."""
    g = gen(41)
    lens = [5000, 0, 9000, 3]
    kc, vc, pt, pl, bt, sl = behind(20000, lens, 64, 2, 64, dtype, g)
    q = randn((4, 16, 64), dtype, g)
    out = check_prefix(q, kc, vc, pt, pl, bt, sl)
    wide = torch.full((pt.numel() + 5000,), -1, dtype=torch.int32, device="cuda")
    wide[:pt.numel()] = pt
    assert torch.equal(la.paged_prefix_decode(q, kc, vc, wide, pl, bt, sl), out)
    own = torch.full((4, 4000), -1, dtype=torch.int32, device="cuda")
    own[:, :bt.shape[1]] = bt
    check_prefix(q, kc, vc, pt, pl, own, ints([1, 2, 0, 3]))
    check_prefix(q, kc, vc, pt, ints([64]), own[:, :3], ints([1, 2, 0, 3]))


def test_prefix_is_the_dense_one():
    g = gen(42)
    page, n, lens = 16, 320, [5, 0, 70]
    kc, vc, pt, pl, bt, sl = behind(n, lens, page, 2, 128, BF16, g)
    q = randn((3, 16, 128), BF16, g)
    out = check_prefix(q, kc, vc, pt, pl, bt, sl).float()
    rows = torch.cat([pt[None, :n // page].expand(3, -1), bt], 1).contiguous()
    dense = la.paged_decode(q, kc, vc, rows, sl + n).float()
    assert ((out - dense).abs() <= 2 ** -7 * dense.abs() + 1e-3).all()  # as for chosen pages


def test_prefix_absent_pages_and_lengths():
    g = gen(43)
    page, lens = 16, [40, 3, 0, 17]
    kc, vc, pt, pl, bt, sl = behind(600, lens, page, 2, 128, BF16, g)
    q = randn((4, 8, 128), BF16, g)
    pt[3], pt[20] = -1, 10 ** 9
    bt[0, 0] = -5
    check_prefix(q, kc, vc, pt, pl, bt, sl)
    pt[16:24] = -1  # a whole tile of 128
    check_prefix(q, kc, vc, pt, pl, bt, sl)
    pt[:] = -1     # nothing is left of the prefix
    out = check_prefix(q, kc, vc, pt, pl, bt, sl)
    assert (out[2] == 0).all()
    check_prefix(q, kc, vc, pt, ints([-3]), bt, sl)
    check_prefix(q, kc, vc, pt[:0], ints([100]), bt, sl)
    good = behind(600, lens, page, 2, 128, BF16, g)
    pt = good[2][:37]  # the table holds 592 tokens of 2^31 - 1
    check_prefix(q, good[0], good[1], pt, ints([2 ** 31 - 1]), good[4], good[5])


@pytest.mark.parametrize("scale", [0.0, -1.0, 3.0])
def test_prefix_scales(scale):
    """A scale of 0 (the mean of the values), a negative one, a large one; a whole tile absent too."""
    g = gen(49)
    kc, vc, pt, pl, bt, sl = behind(400, [20, 0, 3], 16, 2, 128, BF16, g)
    pt[8:16] = -1
    check_prefix(randn((3, 8, 128), BF16, g), kc, vc, pt, pl, bt, sl, scale=scale)


@pytest.mark.parametrize("step", [7, 9, 60, 300])
@pytest.mark.parametrize("batch", [2, 40])
def test_prefix_maximum_that_jumps(step, batch):
    """Tiles of 128 tokens whose scores rise by `step` (in log2) over the ones before, for some
    rows up and for others down."""
    g = gen(50)
    kc, vc, pt, pl, bt, sl = behind(1100, [3] * batch, 16, 1, 64, BF16, g, garbage=0.0)
    t = torch.arange(1100, device="cuda")
    at = (pt[t // 16].long(), 0, t % 16)
    x = kc[at] * 0.1
    x[:, 0] = (t // 128).to(BF16)
    kc[at] = x
    q = randn((batch, 4, 64), BF16, g)
    q[..., 0] = step * torch.tensor([1.0, -1.0, 0.5, 1.0], device="cuda").to(BF16)
    check_prefix(q, kc, vc, pt, pl, bt, sl, scale=math.log(2))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_prefix_of_an_empty_pool(dtype):
    empty = torch.empty((0, 2, 16, 64), dtype=dtype, device="cuda")
    q = randn((3, 4, 64), dtype, gen(51))
    pt, bt = ints([0, 1, 2]), torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    lse = torch.empty((3, 4), device="cuda")
    out = la.paged_prefix_decode(q, empty, empty, pt, ints([40]), bt, ints([5, 0, 32]), lse=lse)
    assert (out == 0).all() and (lse == -INF).all()


@pytest.mark.parametrize("dtype, batch", [(BF16, 3), (BF16, 40), (FP32, 3)])
def test_prefix_large_scores(dtype, batch):
    """Scores in the hundreds that rise or fall along the prefix: the running maximum moves often."""
    g = gen(44)
    lens = [(i * 13) % 50 for i in range(batch)]
    kc, vc, pt, pl, bt, sl = behind(2000, lens, 16, 1, 128, dtype, g, garbage=0.0)
    ramp = torch.linspace(0.1, 9, 2000, device="cuda")
    t = torch.arange(2000, device="cuda")
    at = (pt[t // 16].long(), 0, t % 16)
    kc[at] = (kc[at].float() * ramp[:, None]).to(dtype)
    q = randn((batch, 8, 128), dtype, g)
    check_prefix(q * 3, kc, vc, pt, pl, bt, sl, scale=0.7)
    kc[at] = kc[at].flip(0)
    check_prefix(q, kc, vc, pt, pl, bt, sl, scale=-0.5)


def test_prefix_infinities_that_are_attended_to():
    g = gen(45)
    kc, vc, pt, pl, bt, sl = behind(300, [20] * 3, 16, 1, 128, BF16, g)
    q = randn((3, 4, 128), BF16, g)
    q[..., 0] = q[..., 0].abs() + 1
    # keys of -infinity where every q is positive: weight 0, also for a whole tile and all own tokens
    for t in list(range(128, 256)) + [290]:
        kc[pt[t // 16].long(), 0, t % 16, 0] = -INF
    kc[bt[1, :2].long(), 0, :, 0] = -INF
    good = la.paged_prefix_decode(q, kc, vc, pt, pl, bt, sl)
    left = [t for t in range(300) if not (128 <= t < 256 or t == 290)]
    for r in range(3):
        own = [] if r == 1 else range(20)
        k, v = (torch.cat([torch.stack([x[pt[t // 16].long(), 0, t % 16] for t in left]).cpu()] +
                          [x[bt[r, t // 16].long(), 0, t % 16][None].cpu() for t in own]) for x in (kc, vc))
        want, _, bound, _ = lref.attend(c(q[r]), k, v, 128 ** -0.5, 128)
        ref.within(good[r], want, bound, ref.u_of(BF16), "out")
    # an infinite value makes its column that infinity for all requests, one of another request not
    vc[pt[2].long(), 0, 5, 9] = -INF
    vc[bt[0, 0].long(), 0, 3, 11] = INF
    out = la.paged_prefix_decode(q, kc, vc, pt, pl, bt, sl)
    assert (out[:, :, 9] == -INF).all() and (out[0, :, 11] == INF).all()
    keep = torch.ones(3, 4, 128, dtype=torch.bool, device="cuda")
    keep[:, :, 9] = False
    keep[0, :, 11] = False
    assert torch.equal(out[keep], good[keep])
    # scores that are all -infinity, or one of +infinity or NaN: NaN
    lse = torch.empty((3, 4), device="cuda")
    dead = kc.clone()
    dead[..., 0] = -INF
    out = la.paged_prefix_decode(q, dead, vc, pt, pl, bt, sl, lse=lse)
    assert torch.isnan(out).all() and (lse == -INF).all()
    kc[pt[0].long(), 0, 0, 0] = INF
    assert torch.isnan(la.paged_prefix_decode(q, kc, vc, pt, pl, bt, sl)).all()


def test_prefix_strides_guards_and_refusals():
    g = gen(46)
    kc, vc, pt, pl, bt, sl = behind(130, [65, 200, 9], 16, 2, 64, BF16, g)
    both = torch.stack([kc, vc], dim=1)
    wide = torch.full((3, bt.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.shape[1]] = bt
    x = randn((3, 12, 64), BF16, g)
    buf = torch.full((5, 8, 64), 3.0, dtype=BF16, device="cuda")
    size = la.paged_prefix_decode_workspace_bytes(3, 8, 2, 64)
    ws = torch.full((size + 256,), 77, dtype=torch.uint8, device="cuda")
    out = check_prefix(x[:, :8], both[:, 0], both[:, 1], pt, pl, wide[:, :bt.shape[1]], sl, out=buf[1:4],
                       workspace=ws[:size])
    assert (buf[0] == 3).all() and (buf[4] == 3).all() and (ws[size:] == 77).all()
    assert torch.equal(out, la.paged_prefix_decode(x[:, :8].contiguous(), kc, vc, pt, pl, bt, sl))
    q = x[:, :8]
    for bad in (dict(pt=pt.long()), dict(pt=pt[None]), dict(pl=ints([1, 2])), dict(pl=130), dict(q=x[:, :7]),
                dict(ws=ws[:size - 16]), dict(pt=pt.cpu()), dict(sl=sl[:2]), dict(vc=vc[:, :1])):
        a = {**dict(q=q, kc=kc, vc=vc, pt=pt, pl=pl, sl=sl, ws=None), **bad}
        with pytest.raises((ValueError, TypeError, la.LightningAttnError)):
            la.paged_prefix_decode(a["q"], a["kc"], a["vc"], a["pt"], a["pl"], bt, a["sl"], workspace=a["ws"])
    assert la.paged_prefix_decode(q[:0], kc, vc, pt, pl, bt[:0], sl[:0]).shape == (0, 8, 64)


@pytest.mark.parametrize("batch", [2, 40])
def test_prefix_same_bits_from_a_graph_and_beside_other_calls(batch):
    """Equal calls give equal bits: eager, replayed for other lengths, and two at once on two streams."""
    g = gen(47)
    lens = [(i * 31) % 200 for i in range(batch)]
    kc, vc, pt, pl, bt, sl = behind(9000, lens, 64, 2, 128, BF16, g)
    q = randn((batch, 16, 128), BF16, g)
    want = la.paged_prefix_decode(q, kc, vc, pt, pl, bt, sl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = la.paged_prefix_decode(q, kc, vc, pt, pl, bt, sl)
    for n in (9000, 1, 4444, 0):
        pl.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, check_prefix(q, kc, vc, pt, pl, bt, sl))
    pl.fill_(9000)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(6):
        outs.append(la.paged_prefix_decode(q, kc, vc, pt, pl, bt, sl, stream=streams[i % 2]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_prefix_long_sums_do_not_drift():
    """As for the paged attention: a prefix whose second half has the first one's keys and the negative
    values, the largest scores first.  The formula's output is 0; what remains are additions to a running sum
    below 1.5 sum p, each of which errs by at most 2^-24 of it with either sign where it is rounded to
    nearest.  Additions that drop the excess bits would err to one side, steps 2^-25 in the mean."""
    g = gen(48)
    n, page, d, b = 32768, 64, 128, 64
    k = randn((n // 2, d), FP32, g)
    q = torch.zeros((b, 16, d), device="cuda")
    q[:, :, 0] = 1.0
    k[:, 0] = -k[:, 0].abs()
    k[:256] = 0.0
    v = (0.5 + torch.rand((n // 2, d), generator=g, device="cuda")).to(BF16)
    kc = torch.cat([k, k]).to(BF16).reshape(n // page, 1, page, d)
    vc = torch.cat([v, -v]).reshape(n // page, 1, page, d)
    pt = torch.arange(n // page, dtype=torch.int32, device="cuda")
    bt, lens = torch.zeros((b, 1), dtype=torch.int32, device="cuda"), ints([0] * b)
    out = la.paged_prefix_decode(q.to(BF16), kc, vc, pt, ints([n]), bt, lens, scale=1.0).double()
    steps, samples = n // 16, d
    bound = 10 * math.sqrt(steps) * ref.E * 1.5 / math.sqrt(samples)
    mean = out.mean((0, 1, 2)).abs().item()
    print(f"mean {mean:.3e}, bound {bound:.3e}")
    assert mean <= bound


def test_calls_behind_what_writes_their_arguments():
    """Every argument written by the call right before, in one stream without a wait between: lengths,
    table and slots by the reservation, queries and cache by the append, the choice by the selection."""
    g = gen(52)
    page, hk, h, d, b, count = 16, 2, 16, 128, 6, 9
    pages = 700
    kc, vc = caches(pages, hk, page, d, BF16, g)
    front = torch.arange(600, 640, dtype=torch.int32, device="cuda")
    bd = torch.zeros((pages, hk, 2, d), dtype=BF16, device="cuda")
    table = la.rotary_table(4000, 64, device="cuda")
    xs = [randn((sum(n), h + 2 * hk, d), BF16, g) for n in ([400, 3, 900, 0, 17, 1], [1] * 6, [1] * 6)]

    def loop(wait):
        k, v = kc.clone(), vc.clone()
        bounds = bd.clone()
        bt = torch.full((b, 80), -1, dtype=torch.int32, device="cuda")
        lens, free, top = ints([0] * b), torch.arange(600, dtype=torch.int32, device="cuda"), ints([600])
        got = []
        for new, x in zip(([400, 3, 900, 0, 17, 1], [1] * 6, [1] * 6), xs):
            before = lens.clone()
            slots, pos, cu, _ = la.paged_reserve(bt, lens, ints(new), free, top, page, sum(new))
            wait()
            q = la.paged_append(x[:, :h], x[:, h:h + hk], x[:, h + hk:], pos, table, k, v, slots)
            wait()
            last = (cu[1:] - 1).clamp(min=0).long()
            ql = q[last].contiguous()
            out = la.paged_prefix_decode(ql, k, v, front, ints([630]), bt, lens)
            wait()
            la.paged_bounds(k, bounds, bt, before, lens)
            wait()
            sel = la.paged_select(ql, bounds, bt, lens, page, count)
            wait()
            got += [out, sel, la.paged_sparse_decode(ql, k, v, bt, lens, sel)]
            wait()
            got.append(la.paged_prefix_decode(ql, k, v, front[:0], ints([0]), bt, lens))
            wait()
        return got

    want = loop(torch.cuda.synchronize)
    for _ in range(20):
        assert all(torch.equal(x, y) for x, y in zip(loop(lambda: None), want))


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_serving_loop(dtype):
    """Prompts, then steps: pages reserved, keys appended, bounds kept, pages chosen and attended to.
    Bounds equal those of whole pages taken anew; the rest is as the reference has it."""
    g = gen(31)
    page, hk, h, d, count = 16, 2, 8, 64, 5
    b, pages, width = 4, 120, 30
    kc, vc = caches(pages, hk, page, d, dtype, g)
    bd = torch.full((pages, hk, 2, d), NAN, dtype=dtype, device="cuda")
    bt = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    lens, free, count_ = ints([0] * b), torch.randperm(pages, generator=g, device="cuda").int(), ints([pages])
    table = la.rotary_table(1000, 32, device="cuda")
    w = [1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    for new in ([300, 17, 0, 64], [1, 1, 1, 1], [1, 15, 200, 1], [1, 1, 1, 1]):
        before, fresh, total = lens.clone(), ints(new), sum(new)
        slots, pos, cu, served = la.paged_reserve(bt, lens, fresh, free, count_, page, total)
        assert bool(served.all())
        x = randn((total, h + 2 * hk, d), dtype, g)
        q = la.paged_append(x[:, :h], x[:, h:h + hk], x[:, h + hk:], pos, table, kc, vc, slots,
                            q_weight=w[0], k_weight=w[1])
        la.paged_bounds(kc, bd, bt, before, lens)
        want = lref.bounds(c(kc), c(bd), c(bt), [0] * b, c(lens))
        used = torch.unique(bt[bt >= 0]).long()
        assert torch.equal(bd[used].cpu(), want[used.cpu()])
        last = (cu[1:] - 1).clamp(min=0).long()
        ql = q[last].contiguous()
        sel = check_select(ql, bd, bt, lens, page, count)
        check_sparse(ql, kc, vc, bt, lens, sel)


def run_all(q, kc, vc, bd, bt, first, lens, page, count, **kw):
    la.paged_bounds(kc, bd, bt, first, lens, **kw)
    sel = la.paged_select(q, bd, bt, lens, page, count, **kw)
    return sel, la.paged_sparse_decode(q, kc, vc, bt, lens, sel, **kw)


def test_replayed_from_a_graph_and_on_other_streams():
    g = gen(32)
    lens_list, page, count = [5000, 37, 900], 16, 12
    bt, pages = tables(blocks_of([6000] * 3, page), g)
    kc, vc = caches(pages, 2, page, 128, BF16, g)
    bd0 = torch.zeros((pages, 2, 2, 128), dtype=BF16, device="cuda")
    q, first, lens = randn((3, 16, 128), BF16, g), ints([0, 0, 0]), ints(lens_list)
    want = run_all(q, kc, vc, bd0.clone(), bt, first, lens, page, count)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bd = bd0.clone()
    side.wait_stream(torch.cuda.current_stream())
    got = run_all(q, kc, vc, bd, bt, first, lens, page, count, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph, bd = torch.cuda.CUDAGraph(), bd0.clone()
    with torch.cuda.graph(graph):
        got = run_all(q, kc, vc, bd, bt, first, lens, page, count)
    for seed in (0, 1):  # other lengths and queries, the same graph
        if seed:
            q.copy_(randn(q.shape, BF16, gen(99)))
            lens.copy_(ints([100, 6000, 1]))
            want = run_all(q, kc, vc, bd0.clone(), bt, first, lens, page, count)
        bd.copy_(bd0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_offsets_past_32_bits():
    """More than 2^31 elements of cache, its last pages used."""
    page, hk, d = 64, 8, 128
    pages = 2 ** 31 // (page * hk * d) + 40
    kc = torch.zeros((pages, hk, page, d), dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    g = gen(33)
    kc[-40:] = randn((40, hk, page, d), BF16, g)
    vc[-40:] = randn((40, hk, page, d), BF16, g)
    bd = torch.zeros((pages, hk, 2, d), dtype=BF16, device="cuda")
    bt = torch.arange(pages - 40, pages, dtype=torch.int32, device="cuda")[None]
    q, lens = randn((1, 64, d), BF16, g), ints([40 * page - 5])
    sel, out = run_all(q, kc, vc, bd, bt, ints([0]), lens, page, 9)
    small = bt - (pages - 40)
    bd2 = torch.zeros((40, hk, 2, d), dtype=BF16, device="cuda")
    sel2, out2 = run_all(q, kc[-40:].contiguous(), vc[-40:].contiguous(), bd2, small, ints([0]), lens, page, 9)
    assert torch.equal(sel, sel2) and torch.equal(out, out2) and torch.equal(bd[-40:], bd2)
    own, n = bt[:, :2].contiguous(), ints([70])
    args = [(kc, vc, bt[0, 2:].contiguous(), own), (kc[-40:].contiguous(), vc[-40:].contiguous(),
                                                    small[0, 2:].contiguous(), small[:, :2].contiguous())]
    both = [la.paged_prefix_decode(q, x[0], x[1], x[2], ints([38 * page - 9]), x[3], n) for x in args]
    assert torch.equal(*both)
    assert (bd[:-40] == 0).all()
