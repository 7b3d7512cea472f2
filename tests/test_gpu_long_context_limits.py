"""Long-context operators of the softmax layers at the limits of their contract: calls right behind what
writes their arguments, lengths and values near the types' ends, paths of large calls alone."""
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
    return x.cpu()


# ------------------------------- calls right behind what writes their arguments
def same_behind_their_writers(loop):
    """loop(wait) returns tensors; wait() stands between its kernels.  The same bits with a wait for the GPU
    there, without one, and from a graph that is replayed (no host between two kernels)."""
    want = [x.clone() for x in loop(torch.cuda.synchronize)]
    for _ in range(5):
        got = loop(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = loop(lambda: None)
    for _ in range(10):
        for x in got:
            x.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype, page, width, n", [(BF16, 16, 12, 130), (BF16, 64, 300, 9000), (FP32, 16, 12, 130),
                                                   (FP32, 64, 160, 3000)])
def test_arguments_that_the_kernel_in_front_has_written(dtype, page, width, n):
    """Table, lengths and queries of the choice and of the attention behind a prefix, at one place each, with other
    contents before every call (so that what an earlier call read there is stale), each of them
    in turn the one written last.  Narrow tables (a cluster a unit) and wide ones (split and join)."""
    g = gen(60)
    b, hk, h, d, steps = 5, 2, 16, 128, 6
    pages = 1200
    kc, vc = (randn((pages, hk, page, d), dtype, g) for _ in range(2))
    bd = torch.stack([kc.amin(2), kc.amax(2)], 2)
    sets = []
    for j in range(steps):
        order = torch.randperm(pages, generator=g, device="cuda").int()
        lens = torch.randint(0, n + 1, (b,), generator=g, device="cuda").int()
        lens[j % b] = 0
        sets.append(dict(bt=order[:b * width // 4].repeat(4).reshape(b, width), lens=lens, q=randn((b, h, d), dtype, g),
                         pt=order[-40:].clone(), pl=ints([j * 100 + 37])))
    live = {k: torch.zeros_like(v) for k, v in sets[0].items()}
    names = list(live)

    def loop(wait):
        got = []
        for j, s in enumerate(sets):
            for call in range(2):
                for k in names[j % 5:] + names[:j % 5]:
                    live[k].copy_(s[k])
                wait()
                if call:
                    out = la.paged_select(live["q"], bd, live["bt"], live["lens"], page, 5)
                else:
                    out = la.paged_prefix_decode(live["q"], kc, vc, live["pt"], live["pl"], live["bt"], live["lens"])
                wait()
                got.append(out)
                for k in names:
                    live[k].zero_()
                wait()
        return got

    same_behind_their_writers(loop)


@pytest.mark.parametrize("width", [40, 400])
def test_right_behind_the_reservation_and_the_append(width):
    """The choice and the attention behind a prefix with nothing between them and the reservation (table, lengths) or
    the append (queries, cache); requests end and others take their place, on other pages."""
    g = gen(61)
    page, hk, h, d, b, pages = 16, 2, 16, 128, 6, 500
    kc, vc = (randn((pages, hk, page, d), BF16, g) for _ in range(2))
    bd = torch.stack([kc.amin(2), kc.amax(2)], 2)
    order = torch.randperm(pages - 40, generator=g, device="cuda").int()
    front, length = torch.arange(pages - 40, pages, dtype=torch.int32, device="cuda"), ints([630])
    steps = [([400, 3, 600, 1, 17, 1], [0] * 6), ([1] * 6, [0] * 6), ([1, 30, 1, 200, 1, 1], [0, 1, 1, 0, 0, 0]),
             ([1] * 6, [0] * 6), ([600, 1, 1, 1, 1, 5], [1, 0, 0, 1, 0, 1])]
    steps = [(ints(n), torch.tensor(f, dtype=torch.bool, device="cuda"), sum(n)) for n, f in steps]
    xs = [randn((b, h + 2 * hk, d), BF16, g) for _ in steps]
    q, table = randn((b, h, d), BF16, g), la.rotary_table(1000, 64, device="cuda")
    bt, lens, free, top = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((b, width), b, pages - 40, 1))
    height, k, v, qo = ints([pages - 40]), kc.clone(), vc.clone(), torch.empty_like(q)
    pos = ints([5, 900, 17, 0, 33, 64])
    slots = [(order[-6:] * page + j).contiguous() for j in range(len(steps))]  # pages that are never reserved

    def loop(wait):
        got = []
        bt.fill_(-1), lens.zero_(), free.copy_(order), top.copy_(height)
        k.copy_(kc), v.copy_(vc)
        wait()
        top.sub_(6)
        for (new, over, total), x, at in zip(steps, xs, slots):
            la.paged_reserve(bt, lens, new, free, top, page, total, finished=over)
            wait()
            got.append(la.paged_prefix_decode(q, k, v, front, length, bt, lens))
            wait()
            la.paged_reserve(bt, lens, new, free, top, page, total)
            wait()
            got.append(la.paged_select(q, bd, bt, lens, page, 4))
            wait()
            la.paged_append(x[:, :h], x[:, h:h + hk], x[:, h + hk:], pos, table, k, v, at, q_out=qo)
            wait()
            got.append(la.paged_prefix_decode(qo, k, v, front, length, bt, lens))
            wait()
            la.paged_append(x[:, :h], x[:, h:h + hk], x[:, h + hk:], pos, table, k, v, at, q_out=qo)
            wait()
            got.append(la.paged_select(qo, bd, bt, lens, page, 4))
            wait()
            got += [bt.clone(), lens.clone()]
        return got

    same_behind_their_writers(loop)


# ------------------------------------------------------------ lengths near 2^31
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("page, count", [(1 << 17, 3), (1 << 20, 40)])
def test_chosen_pages_of_the_longest_table(dtype, page, count):
    """A table that holds 2^31 tokens in pages of more than 2^16, most of them absent, and lengths
    that are clamped to what it holds: blocks are counted without passing 32 bits."""
    g = gen(62)
    width, hk, h, d = (1 << 31) // page, 1, 2, 64
    kc, vc = (torch.zeros((2, hk, page, d), dtype=dtype, device="cuda") for _ in range(2))
    for x in (kc, vc):
        x[:, :, :300] = randn((2, hk, 300, d), dtype, g)
        x[:, :, 300:] = NAN
    bt = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    lens = ints([2 ** 31 - 1, 0, 300])
    bt[0, 5], bt[2, 0] = 0, 1  # a full page, whose tokens are all attended to
    kc[0, :, 300:], vc[0, :, 300:] = 0, 0
    sel = torch.full((3, hk, count), -1, dtype=torch.int32, device="cuda")
    sel[0, 0, :3], sel[2, 0, 0] = ints([width - 1, 5, 7]), 0
    q = randn((3, h, d), dtype, g)
    out, lse = torch.full((3, h, d), 7.0, dtype=dtype, device="cuda"), torch.full((3, h), 7.0, device="cuda")
    la.paged_sparse_decode(q, kc, vc, bt, lens, sel, out=out, lse=lse)
    for b, n in ((0, page), (2, 300)):
        at = 0 if b == 0 else 1
        want, wlse, bound, lbound = lref.attend(c(q[b]), c(kc[at, 0, :n]), c(vc[at, 0, :n]), d ** -0.5)
        ref.within(out[b], want, bound, ref.u_of(dtype), "out")
        ref.within(lse[b], wlse, lbound, ref.u_of(FP32), "lse")
    assert (out[1] == 0).all() and (lse[1] == -INF).all()


# ------------------------------------------------- values near the type's largest
@pytest.mark.parametrize("dtype, batch", [(BF16, 2), (BF16, 40), (FP32, 2)])
@pytest.mark.parametrize("step", [3, 3.75, 5, 7.5])
@pytest.mark.parametrize("spike", [True, False])
def test_prefix_large_values_and_scores_that_rise(dtype, batch, step, spike):
    """Scores that rise by `step` (in log2) from one tile of 128 tokens to the next, for one token of it or all, over
    values whose weighted sums against the running maximum are just within the type's range (1.1e38, or
    128 * 1.1e36, and at most 0.6 of it more from other tiles): finite, as the attention without a prefix has it.
    As many key-value heads as there are CTAs, so that each passes about a head's tiles."""
    g = gen(63)
    page, n, hk, group, d = 16, 128 * 12, 152, 4, 64
    t = torch.arange(n, device="cuda")
    score = (t // 128) * step
    v = (0.9 + 0.2 * torch.rand((n, d), generator=g, device="cuda")) * (1e38 if spike else 1e36)
    if spike:  # others are far below the tile's one, and small
        score = torch.where(t % 128 == 77, score, -200.0)
        v[t % 128 != 77] *= 1e-38
    kc, vc = (torch.zeros((n // page + 1, hk, page, d), dtype=dtype, device="cuda") for _ in range(2))
    pt = torch.randperm(n // page, generator=g, device="cuda").int()
    kc[pt[t // page].long(), :, t % page, 0] = score.to(dtype)[:, None]
    vc[pt[t // page].long(), :, t % page] = v.to(dtype)[:, None]
    q = torch.zeros((batch, hk * group, d), dtype=dtype, device="cuda")
    q[..., 0] = torch.tensor([1.0, 1.0, -1.0, 0.5] * hk, device="cuda").to(dtype)
    bt, none = torch.full((batch, 1), n // page, dtype=torch.int32, device="cuda"), ints([0] * batch)
    lse = torch.empty((batch, hk * group), device="cuda")
    out = la.paged_prefix_decode(q, kc, vc, pt, ints([n]), bt, none, scale=math.log(2), lse=lse)
    parts = lref.Behind((c(kc[:, :1]), c(vc[:, :1])), c(pt), n, c(bt[:1]), c(none[:1]))
    want, wlse, bound, lbound = lref.over(c(q[:1, :group]), parts, math.log(2), tile=128)
    assert torch.isfinite(out).all()
    out, lse = out.reshape(batch, hk, group, d), lse.reshape(batch, hk, group)
    for x, y, e, u, name in ((out, want, bound, ref.u_of(dtype), "out"), (lse, wlse, lbound, ref.u_of(FP32), "lse")):
        ref.within(x, y[:, None].expand(x.shape), e[:, None].expand(x.shape), u, name)
    rows = pt[None].expand(batch, -1).contiguous()
    assert torch.isfinite(la.paged_decode(q, kc, vc, rows, none + n, scale=math.log(2))).all()


# --------------------------------------------------------------- a scale of 0
@pytest.mark.parametrize("dtype, batch, d", [(BF16, 3, 128), (BF16, 3, 64), (BF16, 40, 128), (FP32, 3, 64)])
def test_prefix_scale_of_zero_with_infinite_and_nan_queries(dtype, batch, d):
    """0 times an infinite or NaN product is NaN, with own tokens and without; other heads get the mean."""
    g = gen(64)
    page, n, hk, h = 16, 300, 2, 8
    kc, vc = (randn((30, hk, page, d), dtype, g) for _ in range(2))
    pt, bt = torch.arange(20, dtype=torch.int32, device="cuda"), torch.full((batch, 2), 25, dtype=torch.int32, device="cuda")
    own = torch.tensor([0, 7, 0] * batch, dtype=torch.int32, device="cuda")[:batch].contiguous()
    q = randn((batch, h, d), dtype, g)
    bad = torch.zeros((batch, h), dtype=torch.bool, device="cuda")
    for b, head, at, x in ((0, 1, 0, NAN), (0, 5, d - 1, INF), (1, 2, 3, -INF), (2, 7, d // 2, NAN), (batch - 1, 0, 2, INF)):
        q[b, head, at], bad[b, head] = x, True
    lse = torch.empty((batch, h), device="cuda")
    out = la.paged_prefix_decode(q, kc, vc, pt, ints([n]), bt, own, scale=0.0, lse=lse)
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    parts = lref.Behind((c(kc), c(vc)), c(pt), n, c(bt), c(own))
    want, wlse, bound, lbound = lref.over(c(q.masked_fill(bad[..., None], 1.0)), parts, 0.0, tile=128)
    good = ~c(bad)
    ref.within(c(out)[good], want[good], bound[good], ref.u_of(dtype), "out")
    ref.within(c(lse)[good], wlse[good], lbound[good], ref.u_of(FP32), "lse")
    rows = pt[None].expand(batch, -1).contiguous()
    dense = la.paged_decode(q, kc, vc, rows, own * 0 + n, scale=0.0)
    assert torch.isnan(dense[bad]).all() and torch.isfinite(dense[~bad]).all()


# --------------------------------------------------- outputs in place of queries
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("width", [30, 300])
def test_outputs_in_place_of_contiguous_queries(dtype, width):
    """The same bits as in an array of their own; clusters and split with join, several requests in pieces."""
    g = gen(65)
    page, hk, h, d, b = 16, 2, 32, 128, 5
    kc, vc = (randn((900, hk, page, d), dtype, g) for _ in range(2))
    bt = torch.randperm(900, generator=g, device="cuda").int()[:b * width // 3].repeat(3).reshape(b, width)
    lens, pt, pl = ints([width * page, 0, 1, width * 7, width * page - 5]), bt[3, :30].contiguous(), ints([450])
    sel = torch.arange(20, dtype=torch.int32, device="cuda").expand(b, hk, 20).contiguous()
    q = randn((b, h, d), dtype, g)
    for call in (lambda x, **kw: la.paged_decode(x, kc, vc, bt, lens, **kw),
                 lambda x, **kw: la.paged_sparse_decode(x, kc, vc, bt, lens, sel, **kw),
                 lambda x, **kw: la.paged_prefix_decode(x, kc, vc, pt, pl, bt, lens, **kw)):
        want = call(q)
        for _ in range(3):
            x = q.clone()
            assert torch.equal(call(x, out=x), want)
        wide = randn((b, h + 1, d), dtype, g)
        with pytest.raises(la.LightningAttnError, match="in place"):
            call(wide[:, :h], out=wide.flatten()[:b * h * d].view(b, h, d))


# ------------------------------------------------- paths of large calls alone
@pytest.mark.parametrize("dtype, h, hk, d", [(BF16, 8, 2, 64), (BF16, 16, 1, 128), (FP32, 3, 1, 64)])
def test_select_among_more_blocks_than_keys_are_kept(dtype, h, hk, d):
    """8192 blocks' keys stay in shared memory, further ones are made again at every pass: requests on both sides of
    that and far behind it, absent pages among them, few and many equal scores, infinities and NaN."""
    g = gen(66)
    blocks, page = [8192, 8193, 20000, 12288, 9000], 16
    pages = sum(blocks)
    bt = torch.full((5, max(blocks) + 3), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(pages, generator=g, device="cuda").int()
    for b, n in enumerate(blocks):
        bt[b, :n] = order[sum(blocks[:b]):sum(blocks[:b]) + n]
    mid = torch.randn((pages, hk, d), generator=g, device="cuda")
    reach = 0.5 + 2 * torch.rand((pages, hk, d), generator=g, device="cuda")
    bd = torch.stack([mid * 0.5 - reach, mid * 0.5 + reach], 2).to(dtype)
    q = randn((5, h, d), dtype, g)
    lens = ints([n * page - i for i, n in enumerate(blocks)])
    bt[1, 8192], bt[2, 8000:8400], bt[2, 19999] = -1, 10 ** 9, -5
    same = bt[3, 100:12000].long()      # 11900 equal scores, the border among them
    bd[same] = bd[same[:1]]
    bd[bt[4, 8500].long(), 0, 1, 3], bd[bt[4, 8999].long(), 0, 0, 2] = INF, NAN

    def check(count, first, last):
        out = la.paged_select(q, bd, bt, lens, page, count, keep_first=first, keep_last=last)
        assert torch.equal(out.cpu(), lref.select(c(q), c(bd), c(bt), c(lens), page, count, first, last))

    for count, first, last in ((1, 0, 0), (64, 1, 1), (5000, 0, 3), (8192, 1, 0), (12200, 4, 2)):
        check(count, first, last)


@pytest.mark.parametrize("page", [3, 12, 20])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch", [40, 3])
def test_prefix_rows_one_by_one_over_many_tiles(page, d, batch):
    """Pages that no box of eight rows divides, several tiles a CTA and units that begin and end inside its
    range, rows for two groups that share the tiles and for two that do not."""
    g = gen(67)
    n, hk, group = 2900, 24, 8
    pages = -(-n // page) + batch
    kc, vc = (randn((pages, hk, page, d), BF16, g) for _ in range(2))
    pt = torch.randperm(pages - batch, generator=g, device="cuda").int()
    bt = torch.arange(pages - batch, pages, dtype=torch.int32, device="cuda")[:, None].contiguous()
    own = (torch.arange(batch, device="cuda") % (page + 1)).int()
    q = randn((batch, hk * group, d), BF16, g)
    some = [0, 1, 2, 17, 39] if batch == 40 else [0, 1, 2]
    for gone in ([], [0, 7, pt.numel() - 1], list(range(50, 50 + 300 // page))):
        for i in gone:
            pt[i] = -1 if i % 2 else 2 ** 31 - 1
        out = la.paged_prefix_decode(q, kc, vc, pt, ints([n]), bt, own)
        parts = lref.Behind((c(kc), c(vc)), c(pt), n, c(bt[some]), c(own[some]))
        want, _, bound, _ = lref.over(c(q[some]), parts, d ** -0.5, tile=128)
        ref.within(out[some], want, bound, ref.u_of(BF16), "out")


# ------------------------------------------------------ threads, streams, widths
def all_calls(kc, vc, bd, bt, lens, pt, pl, q, page):
    """Every call once, those of a few units and of many; the outputs."""
    b2 = la.paged_bounds(kc, bd.clone(), bt, lens * 0, lens)
    sel = la.paged_select(q, b2, bt, lens, page, 6)
    few = torch.cat([bt, bt[:, :1].expand(-1, 3000) * 0 - 1], 1).contiguous()
    return [b2, sel, la.paged_sparse_decode(q, kc, vc, bt, lens, sel),
            la.paged_prefix_decode(q, kc, vc, pt, pl, bt, lens), la.paged_prefix_decode(q, kc, vc, pt, pl, few, lens),
            la.paged_prefix_decode(q[:1], kc, vc, pt, pl, bt[:1], lens[:1])]


def some_calls(dtype, g, b=20):
    page, hk, h, d = 16, 2, 16, 128
    kc, vc = (randn((400, hk, page, d), dtype, g) for _ in range(2))
    bd = torch.zeros((400, hk, 2, d), dtype=dtype, device="cuda")
    bt = torch.randperm(300, generator=g, device="cuda").int().reshape(b, 300 // b)
    lens, pt, pl = (torch.arange(b, device="cuda") * 11 % 230).int(), torch.arange(300, 400, device="cuda").int(), ints([1590])
    return kc, vc, bd, bt, lens, pt, pl, randn((b, h, d), dtype, g), page


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_two_host_threads(dtype):
    """Calls from two threads, each on its own stream and then both on one: results as alone."""
    import threading
    case = some_calls(dtype, gen(68))
    want = all_calls(*case)
    torch.cuda.synchronize()
    bad, shared = [], torch.cuda.Stream()

    def run(stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = all_calls(*case)
                    stream.synchronize()
                    if not all(torch.equal(x, y) for x, y in zip(got, want)):
                        bad.append("differs")
        except Exception as e:
            bad.append(repr(e))

    for streams in ((torch.cuda.Stream(), torch.cuda.Stream()), (shared, shared)):
        threads = [threading.Thread(target=run, args=(s,)) for s in streams]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    assert not bad, bad


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_streams_inside_a_graph_and_the_default_stream(dtype):
    """Captured calls on two streams that were forked from the capturing one, at once, joined and used; and calls on
    the default stream while another is current."""
    case = some_calls(dtype, gen(69))
    want = [x.clone() for x in all_calls(*case)]
    kc, vc, bd, bt, lens, pt, pl, q, page = case
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = []
        for s in sides:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(all_calls(*case))
        for s in sides:
            torch.cuda.current_stream().wait_stream(s)
        last = la.paged_prefix_decode(q, kc, vc, pt, pl, bt, lens)
    for _ in range(5):
        for x in got[0] + got[1]:
            x.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        for outs in got:
            assert all(torch.equal(x, y) for x, y in zip(outs, want))
        assert torch.equal(last, want[3])
    torch.cuda.synchronize()
    with torch.cuda.stream(sides[0]):
        default = torch.cuda.default_stream()
        out = la.paged_prefix_decode(q, kc, vc, pt, pl, bt, lens, stream=default)
        sel = la.paged_select(q, want[0], bt, lens, page, 6, stream=default)
        few = la.paged_sparse_decode(q, kc, vc, bt, lens, sel, stream=default)
    torch.cuda.synchronize()
    assert torch.equal(out, want[3]) and torch.equal(sel, want[1]) and torch.equal(few, want[2])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_tables_without_a_column(dtype):
    """Requests that can have no token of their own, whatever their lengths say."""
    g = gen(70)
    kc, vc = (randn((40, 2, 16, 64), dtype, g) for _ in range(2))
    bd = torch.zeros((40, 2, 2, 64), dtype=dtype, device="cuda")
    q, lens, none = randn((30, 16, 64), dtype, g), ints([5, 0, -1] * 10), torch.empty((30, 0), dtype=torch.int32, device="cuda")
    assert (la.paged_bounds(kc, bd, none, lens * 0, lens) == 0).all()
    sel = la.paged_select(q, bd, none, lens, 16, 3)
    assert (sel == -1).all()
    lse = torch.zeros((30, 16), device="cuda")
    assert (la.paged_sparse_decode(q, kc, vc, none, lens, sel, lse=lse) == 0).all() and (lse == -INF).all()
    pt, pl = torch.arange(40, dtype=torch.int32, device="cuda"), ints([600])
    out = la.paged_prefix_decode(q, kc, vc, pt, pl, none, lens, lse=lse)
    parts = lref.Behind((c(kc), c(vc)), c(pt), 600, c(none), c(lens))
    want, wlse, bound, lbound = lref.over(c(q), parts, 64 ** -0.5, tile=128)
    ref.within(out, want, bound, ref.u_of(dtype), "out")
    ref.within(lse, wlse, lbound, ref.u_of(FP32), "lse")
    assert (la.paged_prefix_decode(q, kc, vc, none[0], pl, none, lens, lse=lse) == 0).all() and (lse == -INF).all()


def test_writes_are_seen_by_autograd():
    """Calls raise the version of what they write, and of nothing else."""
    kc, vc, bd, bt, lens, pt, pl, q, page = some_calls(BF16, gen(71))
    sel, out = torch.empty((20, 2, 6), dtype=torch.int32, device="cuda"), torch.empty_like(q)
    lse = torch.empty((20, 16), device="cuda")
    every = (kc, vc, bd, bt, lens, pt, pl, q, sel, out, lse)
    for call, written in ((lambda: la.paged_bounds(kc, bd, bt, lens, lens), (bd,)),
                          (lambda: la.paged_select(q, bd, bt, lens, page, 6, out=sel), (sel,)),
                          (lambda: la.paged_sparse_decode(q, kc, vc, bt, lens, sel, out=out, lse=lse), (out, lse)),
                          (lambda: la.paged_prefix_decode(q, kc, vc, pt, pl, bt, lens, out=out, lse=lse), (out, lse))):
        before = [x._version for x in every]
        call()
        for x, v in zip(every, before):
            assert (x._version > v) == any(x is y for y in written)
