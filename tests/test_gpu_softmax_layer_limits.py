"""Softmax-layer operators at the edges of their contracts, against the 64-bit
reference (softmax_reference.py, which derives the bounds): sums over long
caches, infinities in rows that are attended to, token totals past 32 bits,
streams other than the current one, and the paths that only large calls take."""
import math

import pytest
import torch

import softmax_reference as ref
import lightning_attention_attn_gb300 as la
from lightning_attention_attn_gb300 import build as labuild

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
EPS = 1e-6
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


# ------------------------------------------------------- sums over a long cache
@pytest.mark.parametrize("d, h", [(128, 8), (64, 8), (128, 16)])
def test_long_sums_do_not_drift(d, h):
    """A cache whose second half repeats the first one's keys with the values negated: the
    formula's output is 0, the sum of weighted values rises and falls again.  The first
    tokens have the largest scores, so both halves get the same weights and each group's
    products cancel exactly; what remains are the additions to a running sum that stays
    below half of sum p |v| <= 1.5 sum p.  Rounded to nearest, an addition errs by at most
    2^-24 of that with either sign: `steps` of them, in `samples` outputs of other values,
    have a mean of standard deviation below sqrt(steps) 2^-24 1.5 / sqrt(samples); 10 of them are
    allowed.  (Additions that drop the excess bits err to one side, steps 2^-25 in the mean.)"""
    g = gen(d + h)
    n, page, b = 32768, 64, 304  # as many requests as the work has parts; all read the same pages
    k = randn((n // 2, d), FP32, g)
    q = torch.full((b, h, d), 0.0, device="cuda")
    q[:, :, 0] = 1.0
    k[:, 0] = -k[:, 0].abs()
    k[:256] = 0.0
    v = (0.5 + torch.rand((n // 2, d), generator=g, device="cuda")).to(BF16)
    kc = torch.cat([k, k]).to(BF16).reshape(n // page, 1, page, d)
    vc = torch.cat([v, -v]).reshape(n // page, 1, page, d)
    bt = torch.arange(n // page, dtype=torch.int32, device="cuda")[None].repeat(b, 1)
    out = la.paged_decode(q.to(BF16), kc, vc, bt, ints([n] * b), scale=1.0).double()
    steps, samples = n // 16 // 4, d  # a warp's; requests and heads repeat the same sums
    bound = 10 * math.sqrt(steps) * ref.E * 1.5 / math.sqrt(samples)
    mean = out.mean((0, 1, 2)).abs().item()
    print(f"mean {mean:.3e}, bound {bound:.3e}")
    assert mean <= bound


# ------------------------------------------------------------- page reservation
@pytest.mark.parametrize("num_tokens", [16, 4096, 4097, 5016])
@pytest.mark.parametrize("in_place", [True, False])
def test_paged_reserve_total_past_32_bits(num_tokens, in_place):
    """A refused request of nearly 2^31 tokens before a served one: the pages, slots and lengths
    are those of the requests themselves, and the offsets stop at 2^31 - 1."""
    page, width, pages = 16, 400, 1000
    table = torch.full((4, width), -7, dtype=torch.int32, device="cuda")
    lens, new = ints([0, 3, 20, 0]), ints([5000, 2 ** 31 - 1, 16, 2 ** 31 - 1])
    table[1, 0], table[2, :2] = 998, ints([996, 997])
    stack, count = torch.arange(pages, device="cuda").int(), ints([990])
    out = {} if in_place else dict(seq_lens_out=torch.empty_like(lens), free_count_out=torch.empty_like(count))
    slots, pos, cu, served = la.paged_reserve(table, lens, new, stack, count, page, num_tokens, **out)
    assert served.tolist() == [True, False, True, False]
    assert out.get("seq_lens_out", lens).tolist() == [5000, 3, 36, 0]
    assert out.get("free_count_out", count).tolist() == [990 - 313 - 1]
    assert stack.tolist() == list(range(pages))
    want = torch.full((4, width), -7)
    want[0, :313] = 989 - torch.arange(313)  # from the top of the stack
    want[1, 0] = 998
    want[2, :3] = torch.tensor([996, 997, 989 - 313])
    assert torch.equal(table.cpu(), want.int())
    assert cu.tolist() == [0, 5000, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]
    t = torch.arange(num_tokens)
    mine = t < 5000
    assert torch.equal(pos.cpu(), torch.where(mine, t, 0).int())
    rows = want[0, (t // page).clamp(max=312)] * page + t % page
    assert torch.equal(slots.cpu(), torch.where(mine, rows, -1).int())


# ------------------------------------------------ infinities that are attended to
def attend(q, kc, vc, bt, lens, out, lse, without=()):
    """Checks out and lse: NaN and infinities where the formula has them, the rest within
    the bounds.  without: (request, block) that the reference leaves out, for keys whose
    score is -infinity (weight 0), which would make the bound itself infinite."""
    left = bt.clone()
    for b, blk in without:
        left[b, blk] = -1
    want, wlse, bound, lbound = ref.attention(q.cpu(), kc.cpu(), vc.cpu(), left.cpu(), lens.cpu(),
                                              q.shape[-1] ** -0.5)
    out, lse = out.cpu().double(), lse.cpu().double()
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    some = ~torch.isnan(want)
    bound = torch.where(torch.isfinite(want), bound, torch.zeros_like(bound))
    ref.within(out[some], want[some], bound[some], ref.u_of(vc.dtype), "out")
    some = ~torch.isnan(wlse)
    ref.within(lse[some], wlse[some], lbound[some], ref.u_of(FP32), "lse")
    return want


def caches(lens, page, hk, d, dtype, g):
    blocks = [-(-n // page) for n in lens]
    kc, vc = (randn((sum(blocks) + 1, hk, page, d), dtype, g) for _ in range(2))
    bt = torch.full((len(lens), max(blocks)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(blocks):
        bt[b, :n] = torch.arange(at, at + n)
        at += n
    return kc, vc, bt, ints(lens)


def widened(bt, width):
    wide = torch.full((bt.shape[0], width), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.shape[1]] = bt
    return wide


SHAPES = [(BF16, 128, 8, 1), (BF16, 64, 12, 1), (BF16, 64, 4, 2), (BF16, 128, 32, 2), (FP32, 64, 6, 2),
          (FP32, 128, 16, 1)]


@pytest.mark.parametrize("wide", [False, True])  # one cluster a unit; the split over all CTAs
@pytest.mark.parametrize("dtype, d, h, hk", SHAPES)
def test_infinite_values(dtype, d, h, hk, wide):
    """Infinite values among those attended to: their column is that infinity for every head,
    or NaN where both signs or a NaN meet; the other columns are what they are without it.
    Scores are small, so that every weight is a normal number."""
    g = gen(d + h)
    lens = [700, 33, 1, 2000]
    kc, vc, bt, sl = caches(lens, 16, hk, d, dtype, g)
    v = vc[:, 0]
    v[bt[0, 3], 5, 7] = INF
    v[bt[0, 40], 1, 9] = -INF
    v[bt[0, 1], 2, 11], v[bt[0, 30], 2, 11] = INF, -INF
    v[bt[1, 2], 0, 0] = -INF
    v[bt[2, 0], 0, d - 1] = INF
    v[bt[3, 100], 8, 20] = NAN
    q = randn((4, h, d), dtype, g)
    table = widened(bt, 20000) if wide else bt
    lse = torch.empty((4, h), device="cuda")
    out = la.paged_decode(q, kc, vc, table, sl, lse=lse)
    want = attend(q, kc, vc, bt, sl, out, lse)
    assert torch.isinf(want[0, 0, 7]) and torch.isnan(want[0, 0, 11]) and torch.isfinite(want[0, 0, 8])
    # the fused step of the same caches
    k1, v1 = kc[bt[:, 0].long(), :, 0].contiguous(), vc[bt[:, 0].long(), :, 0].contiguous()
    out = la.paged_step(q, k1, v1, None, None, kc, vc, bt[:, 0] * 16, table, sl, lse=lse)
    attend(q, kc, vc, bt, sl, out, lse)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype, d, h, hk", SHAPES)
def test_infinite_keys(dtype, d, h, hk, wide):
    """A key with an infinity has the score -infinity (weight 0) for queries of one sign there and
    +infinity (NaN) for the other: the same in paged_decode and in paged_step, whose queries
    are fp32."""
    g = gen(d + h + 1)
    lens = [600, 17, 40]
    kc, vc, bt, sl = caches(lens, 1, hk, d, dtype, g)  # a page a token: the reference can leave it out
    kc[bt[0, 100], :, 0, 3] = -INF
    kc[bt[0, 500], :, 0, 3] = -INF
    kc[bt[1, 16], :, 0, 3] = -INF
    q = randn((3, h, d), dtype, g)
    q[:, :, 3] = q[:, :, 3].abs() + 0.5
    gone = [(0, 100), (0, 500), (1, 16)]
    table = widened(bt, 300000) if wide else bt
    lse = torch.empty((3, h), device="cuda")
    weight = 1 + 0.25 * torch.rand(d, generator=g, device="cuda")  # queries that are no bf16 numbers
    k1, v1 = kc[bt[:, 0].long(), :, 0].contiguous(), vc[bt[:, 0].long(), :, 0].contiguous()
    args = dict(q_weight=weight, k_weight=torch.ones(d, device="cuda"), eps=EPS)
    for sign in (1, -1):
        q[0, 0, 3] = sign * q[0, 0, 3].abs()  # one head that sees +infinity at the second turn
        out = la.paged_decode(q, kc, vc, table, sl, lse=lse)
        want = attend(q, kc, vc, bt, sl, out, lse, gone) if sign > 0 else None
        step = la.paged_step(q, k1, v1, None, None, kc, vc, bt[:, 0].contiguous(), table, sl, lse=lse, **args)
        rotated, _ = ref.norm_rope(q.cpu(), weight.cpu(), EPS, None, None, False)
        want, wlse, bound, _ = ref.attention(rotated, kc.cpu(), vc.cpu(), _left(bt, gone).cpu(), sl.cpu(),
                                             d ** -0.5)
        # 2^-16 of an element for split queries, their own 64 e beside it: see test_paged_step
        more = 1 + (2.0 ** -16 + 128 * ref.E) / (2 * ref.E * (d + 8))
        some = torch.ones(3, h, dtype=torch.bool)
        if sign < 0:
            some[0, 0] = False
            assert torch.isnan(out[0, 0]).all() and torch.isnan(step[0, 0]).all()
        ref.within(step.cpu()[some], want[some], bound[some] * more, ref.u_of(dtype), "step")
        assert torch.isfinite(out.cpu()[some]).all()


def _left(bt, gone):
    left = bt.clone()
    for b, blk in gone:
        left[b, blk] = -1
    return left


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype, d, h, hk", SHAPES)
def test_scores_that_are_all_minus_infinity(dtype, d, h, hk, wide):
    """0 / 0: NaN, with -infinity as the logarithm of the sum; zeros only where there is no
    token.  A finite score anywhere makes the others weight 0."""
    g = gen(d + h + 2)
    lens = [300, 1, 0, 513, 40]
    kc, vc, bt, sl = caches(lens, 16, hk, d, dtype, g)
    q = randn((5, h, d), dtype, g)
    q[:, :, 3] = 1.0
    for b, n in ((0, 300), (1, 1), (3, 513)):
        kc[bt[b, :-(-n // 16)].long(), :, :, 3] = -INF
    kc[bt[3, 32], :, 0, 3] = 0.25          # request 3: its last token alone counts
    bt[4] = -1                              # request 4: no page is left
    table = widened(bt, 20000) if wide else bt
    lse = torch.empty((5, h), device="cuda")
    out = la.paged_decode(q, kc, vc, table, sl, lse=lse)
    assert torch.isnan(out[:2]).all() and (lse[:2] == -INF).all()
    assert (out[2] == 0).all() and (lse[2] == -INF).all()
    assert (out[4] == 0).all() and (lse[4] == -INF).all()
    only = vc[bt[3, 32].long(), :, 0].repeat_interleave(h // hk, 0)
    assert torch.equal(out[3], only)


# ------------------------------------------------------------------- streams
def busy(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(200_000_000)  # about 0.1 s


def test_outputs_and_inputs_of_a_call_on_another_stream():
    """Memory of a call on a stream that is not the current one is not handed out again
    while either stream still has to use it."""
    g = gen(30)
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    n, h, d = 1031, 16, 128  # a size that nothing else has
    x = randn((n, h, d), BF16, g)
    la.qk_norm_rope(x, None, stream=side)
    torch.cuda.synchronize()

    # the output: dropped while the current stream has yet to read it
    out, _ = la.qk_norm_rope(x, None, stream=side)
    here.wait_stream(side)
    busy(here)
    copy = out.clone()
    at, want = out.data_ptr(), x.clone()
    del out
    with torch.cuda.stream(side):
        again = torch.empty((n, h, d), dtype=BF16, device="cuda")
    assert again.data_ptr() != at
    again, _ = la.qk_norm_rope(torch.zeros_like(x), None, stream=side)
    assert again.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
    del again, copy

    # an input: dropped while the call has yet to run
    y = x.clone()
    side.wait_stream(here)
    busy(side)
    out, _ = la.qk_norm_rope(y, None, stream=side)
    at = y.data_ptr()
    del y
    assert torch.empty((n, h, d), dtype=BF16, device="cuda").data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(out, x)


def test_streams_inside_a_graph_and_the_default_stream():
    """A captured call on a stream that was forked from the capturing one, its output used and
    dropped inside the capture; and the default stream named while another one is current."""
    g = gen(32)
    kc, vc, bt, sl = caches([5000, 40, 0, 900], 16, 2, 64, BF16, g)
    vc[bt[0, 100], 0, 3, 5] = INF
    table = widened(bt, 4096)
    q = randn((4, 8, 64), BF16, g)
    want = la.paged_decode(q, kc, vc, table, sl)
    side, own = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        outs = []
        for _ in range(3):
            side.wait_stream(here)
            out = la.paged_decode(q, kc, vc, table, sl, stream=side)
            here.wait_stream(side)
            outs.append(out.clone())
            del out
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
    for o in outs:
        assert torch.equal(o, want)
    default = torch.cuda.default_stream()
    with torch.cuda.stream(own):
        x = q + 0
        default.wait_stream(own)
        out = la.paged_decode(x, kc, vc, table, sl, stream=default)
        own.wait_stream(default)
        del x
        got = out.clone()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.isinf(want[0, 0, 5])


# ------------------------------------------------------- what autograd is told
def test_writes_are_seen_by_autograd():
    g = gen(31)
    h, hk, d, page = 4, 2, 64, 16
    q, k, v = (randn((2, n, d), BF16, g) for n in (h, hk, hk))
    kc, vc = (randn((6, hk, page, d), BF16, g) for _ in range(2))
    bt, lens, new = ints([[0, 1], [2, 3]]), ints([20, 17]), ints([1, 1])
    stack, count = ints([4, 5, 0, 0, 0, 0]), ints([2])
    out, lse = torch.empty_like(q), torch.empty((2, h), device="cuda")
    qo, ko, dq, dk = (torch.empty_like(z) for z in (q, k, q, k))
    lo, co = torch.empty_like(lens), torch.empty_like(count)

    def raised(f, written, kept):
        before = [t._version for t in (*written, *kept)]
        f()
        after = [t._version for t in (*written, *kept)]
        assert all(a > b for a, b in zip(after[:len(written)], before))
        assert after[len(written):] == before[len(written):]

    w = torch.ones(d, device="cuda")
    slots = ints([19, 48])
    raised(lambda: la.qk_norm_rope(q, k, q_out=qo, k_out=ko), (qo, ko), (q, k))
    raised(lambda: la.qk_norm_rope(q, k, q_out=q, k_out=k), (q, k), ())
    raised(lambda: la.qk_norm_rope_backward(q, k, None, None, qo, ko, q_weight=w, k_weight=w, dq=dq, dk=dk),
           (dq, dk), (q, k, qo, ko, w))
    raised(lambda: la.paged_append(q, k, v, None, None, kc, vc, slots, q_out=qo), (kc, vc, qo), (q, k, v, slots))
    raised(lambda: la.paged_decode(q, kc, vc, bt, lens, out=out, lse=lse), (out, lse), (q, kc, vc, bt, lens))
    raised(lambda: la.paged_step(q, k, v, None, None, kc, vc, slots, bt, lens, out=out, lse=lse),
           (kc, vc, out, lse), (q, k, v, bt, lens))
    raised(lambda: la.paged_reserve(bt, lens, new, stack, count, page, 2, seq_lens_out=lo, free_count_out=co),
           (bt, stack, lo, co), (lens, new, count))
    raised(lambda: la.paged_reserve(bt, lens, new, stack, count, page, 2), (bt, stack, lens, count), (new,))

    # a saved input that is overwritten: an error instead of a wrong gradient
    a = torch.ones((2, h, d), device="cuda", requires_grad=True)
    b = a * 2
    c = b * b
    la.qk_norm_rope(b.detach(), None, q_weight=w, q_out=b.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        c.sum().backward()
    # tensors without a version are written all the same
    with torch.inference_mode():
        t = q.clone()
        la.qk_norm_rope(t, None, q_weight=w, q_out=t)
    la.qk_norm_rope(t, None, q_weight=w, q_out=t)


# ------------------------------------------------- paths of large calls alone
@pytest.mark.parametrize("dtype, t, h, hk, d, rot, inter", [
    (BF16, 700, 64, 64, 64, 64, False), (BF16, 500, 64, 64, 64, 32, True), (BF16, 600, 64, 16, 128, 64, False),
    (BF16, 600, 64, 16, 128, 128, True), (BF16, 300, 96, 32, 128, 48, True), (FP32, 500, 64, 64, 128, 128, False),
    (FP32, 500, 64, 64, 128, 64, True), (FP32, 700, 64, 64, 64, 64, True), (FP32, 700, 64, 64, 64, 48, False),
    (BF16, 700, 33, 17, 64, 32, False), (FP32, 700, 33, 17, 128, 16, True)])
def test_norm_rope_of_many_rows(dtype, t, h, hk, d, rot, inter):
    """Forward and gradients where a warp takes several passes, for every type, width and rotation;
    heads that fill its passes (no checks inside) and heads that do not."""
    assert t * (h + hk) > 152 * 16 * (32 // (d // 8))  # above the limit of single passes
    g = gen(t + d + rot)
    x = randn((t, h + hk, d), dtype, g)
    q, k = x[:, :h], x[:, h:]
    w = [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    table = la.rotary_table(5000, rot, device="cuda")
    pos = torch.randint(0, 5000, (t,), generator=g, device="cuda", dtype=torch.int32)
    args = dict(q_weight=w[0], k_weight=w[1], eps=EPS, interleaved=inter)
    outs = la.qk_norm_rope(q, k, pos, table, **args)
    dy = [randn(z.shape, dtype, g) for z in (q, k)]
    grads = la.qk_norm_rope_backward(q, k, pos, table, *dy, **args)
    for i, z in enumerate((q, k)):
        a = (z.cpu(), w[i].cpu(), EPS, table.cpu(), pos.cpu(), inter)
        want, bound = ref.norm_rope(*a)
        ref.within(outs[i], want, bound, ref.u_of(dtype), "y")
        want, wantw, bound, boundw = ref.norm_rope_backward(*a, dy[i].cpu())
        ref.within(grads[i], want, bound, ref.u_of(dtype), "dx")
        ref.within(grads[2 + i], wantw, boundw, ref.u_of(FP32), "dw")


@pytest.mark.parametrize("dtype, b, h, hk, d, rot, inter", [
    (BF16, 128, 64, 8, 128, 64, False), (BF16, 200, 64, 8, 64, 64, True), (BF16, 300, 24, 1, 128, 32, True),
    (FP32, 128, 64, 8, 128, 128, False), (FP32, 140, 48, 12, 64, 16, False)])
def test_paged_step_of_a_full_batch(dtype, b, h, hk, d, rot, inter):
    """Steps whose queries pass from one half to the other out of warps that take several passes."""
    assert b * (h + 2 * hk) > 152 * 16 * (32 // (d // 8))
    g = gen(b + d)
    page, most = 16, 150
    lens = torch.randint(1, most, (b,), generator=g, device="cuda", dtype=torch.int32)
    blocks = -(-most // page)
    kc, vc = (randn((b * blocks, hk, page, d), dtype, g) for _ in range(2))
    bt = torch.randperm(b * blocks, generator=g, device="cuda").int().reshape(b, blocks)
    x = randn((b, h + 2 * hk, d), dtype, g)
    q, k, v = x[:, :h], x[:, h:h + hk], x[:, h + hk:]
    w = [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    table = la.rotary_table(most, rot, device="cuda")
    pos = lens - 1
    slots = bt.gather(1, (pos // page)[:, None].long())[:, 0] * page + pos % page
    args = dict(q_weight=w[0], k_weight=w[1], eps=EPS, interleaved=inter)
    lse = torch.empty((b, h), device="cuda")
    out = la.paged_step(q, k, v, pos, table, kc, vc, slots, bt, lens, lse=lse, **args)
    at = (slots // page).long(), slice(None), (slots % page).long()
    assert torch.equal(vc[at], v)
    want, bound = ref.norm_rope(k.cpu(), w[1].cpu(), EPS, table.cpu(), pos.cpu(), inter)
    ref.within(kc[at], want, bound, ref.u_of(dtype), "key")
    rotated, qbound = ref.norm_rope(q.cpu(), w[0].cpu(), EPS, table.cpu(), pos.cpu(), inter)
    want, wlse, bound, lbound = ref.attention(rotated, kc.cpu(), vc.cpu(), bt.cpu(), lens.cpu(), d ** -0.5)
    # the queries' own fp32 error and their split into two bf16 parts, as in test_paged_step
    extra = (qbound / rotated.abs().amax(-1, keepdim=True).clamp(min=1e-3)).amax() + 2.0 ** -16
    more = 1 + float(extra) / (2 * ref.E * (d + 8))
    ref.within(out, want, bound * more, ref.u_of(dtype), "out")
    ref.within(lse, wlse, lbound * more, ref.u_of(FP32), "lse")


@pytest.mark.parametrize("dtype, hk, empty", [(BF16, 1, 0), (FP32, 2, 0), (BF16, 2, 3000), (FP32, 1, 700)])
def test_more_requests_than_a_block_has_threads(dtype, hk, empty):
    """Hundreds of requests, long ones among them at the ends and in the middle, so that the pieces of
    cut units are joined from several rounds of the prefix sums; optionally with thousands
    without tokens in between."""
    g = gen(hk + empty)
    h, d, page = 8 * hk, 64, 64
    long = {0: 9000, 149: 3000, 299: 5000, 599: 7001}
    lens_list = [long.get(i, 1 + i % 40) for i in range(300)] + [0] * empty + \
        [long.get(i, 1 + i % 40) for i in range(300, 600)]
    b = len(lens_list)
    pages = 160
    kc, vc = (randn((pages, hk, page, d), dtype, g) for _ in range(2))
    bt = torch.randint(0, pages, (b, 9000 // page + 2000), generator=g, device="cuda", dtype=torch.int32)
    q = randn((b, h, d), dtype, g)
    lens, lse = ints(lens_list), torch.empty((b, h), device="cuda")
    out = la.paged_decode(q, kc, vc, bt, lens, lse=lse)
    want, wlse, bound, lbound = ref.attention(q.cpu(), kc.cpu(), vc.cpu(), bt.cpu(), lens.cpu(), d ** -0.5)
    ref.within(out, want, bound, ref.u_of(dtype), "out")
    ref.within(lse, wlse, lbound, ref.u_of(FP32), "lse")
