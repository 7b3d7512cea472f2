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
    assert (bd[:-40] == 0).all()
