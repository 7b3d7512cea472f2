"""GPU parity of the softmax layers' operators against the 64-bit reference
(softmax_reference.py, which derives the bounds), at the sizes, strides and
masks where they can go wrong; a serving loop and a training pass of them
together."""

import pytest
import torch

import oracle
import softmax_reference as ref
import lightning_attention_attn_gb300 as la
from lightning_attention_attn_gb300 import build as labuild
from lightning_attention_attn_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
EPS = 1e-6


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


def qkv(t, h, hk, d, dtype, g):
    """Slices of one fused projection."""
    x = randn((t, h + 2 * hk, d), dtype, g)
    return x[:, :h], x[:, h:h + hk], x[:, h + hk:]


def weights(d, g):
    return [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]


def positions_of(t, rows, g):
    return torch.randint(0, rows, (t,), generator=g, device="cuda", dtype=torch.int32)


def c(x):
    return None if x is None else x.cpu()


# --------------------------------------------------------- norm + rotation
NORM_CASES = [
    # dtype, tokens, heads, kv heads, head_dim, rotary_dim, interleaved, norm
    (BF16, 1, 64, 8, 128, 64, False, True),
    (BF16, 1, 1, 1, 64, 64, False, True),
    (BF16, 3, 7, 3, 128, 128, True, True),
    (BF16, 65, 12, 4, 64, 32, False, True),
    (BF16, 33, 5, 0, 128, 16, True, True),
    (BF16, 700, 64, 64, 128, 128, False, True),    # enough rows for four passes a warp
    (BF16, 17, 6, 2, 128, 0, False, True),
    (BF16, 17, 6, 2, 64, 48, False, False),
    (FP32, 1, 3, 1, 64, 64, False, True),
    (FP32, 31, 5, 2, 128, 96, True, True),
    (FP32, 40, 4, 4, 128, 112, False, True),
    (FP32, 1021, 12, 4, 64, 64, True, True),
    (FP32, 9, 2, 1, 64, 16, False, False),
]


def norm_inputs(case, seed):
    dtype, t, h, hk, d, rot, interleaved, norm = case
    g = gen(seed)
    q, k, _ = qkv(t, h, hk, d, dtype, g)
    k = k if hk else None
    qw, kw = weights(d, g) if norm else (None, None)
    kw = kw if hk else None
    table = la.rotary_table(5000, rot, device="cuda") if rot else None
    pos = positions_of(t, 5000, g) if rot else None
    return g, q, k, qw, kw, pos, table


@pytest.mark.parametrize("case", NORM_CASES, ids=str)
def test_qk_norm_rope(case):
    dtype, inter = case[0], case[6]
    _, q, k, qw, kw, pos, table = norm_inputs(case, 1)
    qo, ko = la.qk_norm_rope(q, k, pos, table, q_weight=qw, k_weight=kw, eps=EPS, interleaved=inter)
    for x, w, got, name in ((q, qw, qo, "q"), (k, kw, ko, "k")):
        if x is None:
            assert got is None
            continue
        want, bound = ref.norm_rope(c(x), c(w), EPS, c(table), c(pos), inter)
        ref.within(got, want, bound, ref.u_of(dtype), name)


@pytest.mark.parametrize("case", NORM_CASES, ids=str)
def test_qk_norm_rope_backward(case):
    dtype, t, h, hk, d, _, inter, norm = case
    g, q, k, qw, kw, pos, table = norm_inputs(case, 2)
    dqo = randn(q.shape, dtype, g)
    dko = randn(k.shape, dtype, g) if hk else None
    args = dict(q_weight=qw, k_weight=kw, eps=EPS, interleaved=inter)
    got = la.qk_norm_rope_backward(q, k, pos, table, dqo, dko, **args)
    for x, w, dy, dx, dw, name in ((q, qw, dqo, got[0], got[2], "q"),
                                   (k, kw, dko, got[1], got[3], "k")):
        if x is None:
            assert dx is None and dw is None
            continue
        want, wantw, bound, boundw = ref.norm_rope_backward(c(x), c(w), EPS, c(table), c(pos), inter,
                                                            c(dy))
        ref.within(dx, want, bound, ref.u_of(dtype), "d" + name)
        if norm:
            ref.within(dw, wantw, boundw, ref.u_of(FP32), f"d{name} weight")
        else:
            assert dw is None
    again = la.qk_norm_rope_backward(q, k, pos, table, dqo, dko, **args)
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)


def test_norm_rope_gradient_against_differences():
    """The fp32 gradients as slopes of the 64-bit forward form."""
    case = (FP32, 5, 3, 2, 64, 32, False, True)
    g, q, k, qw, kw, pos, table = norm_inputs(case, 3)
    dqo, dko = randn(q.shape, FP32, g), randn(k.shape, FP32, g)
    dq, _, dqw, _ = la.qk_norm_rope_backward(q, k, pos, table, dqo, dko, q_weight=qw, k_weight=kw,
                                             eps=EPS)

    def loss(x, w):
        return float((ref.norm_rope(x, w, EPS, c(table), c(pos), False)[0] * c(dqo).double()).sum())

    x, w, step = c(q).double(), c(qw).double(), 1e-6
    cpu = torch.Generator().manual_seed(1)
    for at, grad in ((0, dq), (1, dqw)):
        way = torch.randn(grad.shape, generator=cpu, dtype=torch.float64)
        ends = [loss(*((x + s * way, w) if at == 0 else (x, w + s * way))) for s in (step, -step)]
        slope = (ends[0] - ends[1]) / (2 * step)
        got = c(grad).double()
        # the gradient's fp32 rounding over all elements; differences are exact to 1e-8 here
        room = 128 * ref.E * float((got.abs().mean() + 1) * way.abs().sum()) + 1e-6
        assert abs(slope - float((got * way).sum())) <= room


def test_norm_rope_in_place_and_strided_outputs():
    case = (BF16, 37, 8, 2, 128, 64, False, True)
    g, q, k, qw, kw, pos, table = norm_inputs(case, 4)
    args = dict(q_weight=qw, k_weight=kw, eps=EPS)
    want = la.qk_norm_rope(q, k, pos, table, **args)
    dqo, dko = randn(q.shape, BF16, g), randn(k.shape, BF16, g)
    grads = la.qk_norm_rope_backward(q, k, pos, table, dqo, dko, **args)
    # gradients into the slices of a fused one, and over their own inputs
    fused = torch.full((37, 12, 128), 7.0, dtype=BF16, device="cuda")
    la.qk_norm_rope_backward(q, k, pos, table, dqo, dko, dq=fused[:, :8], dk=fused[:, 8:10], **args)
    assert torch.equal(fused[:, :8], grads[0]) and torch.equal(fused[:, 8:10], grads[1])
    assert (fused[:, 10:] == 7).all()
    la.qk_norm_rope_backward(q, k, pos, table, dqo, dko, dq=dqo, dk=dko, **args)
    assert torch.equal(dqo, grads[0]) and torch.equal(dko, grads[1])
    la.qk_norm_rope(q, k, pos, table, q_out=q, k_out=k, **args)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.parametrize("dtype, inter", [(BF16, False), (BF16, True), (FP32, False)])
def test_norm_rope_in_place_many_rows(dtype, inter):
    """In place where a warp has many passes in flight, heads that end inside one."""
    case = (dtype, 900, 37, 5, 64, 32, inter, True)
    g, q, k, qw, kw, pos, table = norm_inputs(case, 6)
    args = dict(q_weight=qw, k_weight=kw, eps=EPS, interleaved=inter)
    dqo, dko = randn(q.shape, dtype, g), randn(k.shape, dtype, g)
    want = la.qk_norm_rope(q, k, pos, table, **args)
    grads = la.qk_norm_rope_backward(q, k, pos, table, dqo, dko, **args)
    la.qk_norm_rope_backward(q, k, pos, table, dqo, dko, dq=dqo, dk=dko, **args)
    assert torch.equal(dqo, grads[0]) and torch.equal(dko, grads[1])
    la.qk_norm_rope(q, k, pos, table, q_out=q, k_out=k, **args)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_norm_rope_edges():
    g = gen(5)
    table = la.rotary_table(100, 64, device="cuda")
    w = weights(64, g)
    q, k, _ = qkv(4, 2, 1, 64, BF16, g)
    # positions outside the table are clamped to it
    far = torch.tensor([-5, 99, 100, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    near = torch.tensor([0, 99, 99, 99], dtype=torch.int32, device="cuda")
    a = la.qk_norm_rope(q, k, far, table, q_weight=w[0], k_weight=w[1])
    b = la.qk_norm_rope(q, k, near, table, q_weight=w[0], k_weight=w[1])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # without a norm: an infinity or NaN stays with its rotated pair
    x = q.clone()
    x[0, 0, 50], x[1, 1, 3] = float("inf"), float("nan")
    half = la.rotary_table(100, 32, device="cuda")
    out, _ = la.qk_norm_rope(x, None, near, half)
    want, bound = ref.norm_rope(c(q), None, 0, c(half), c(near), False)
    bad = torch.zeros(4, 2, 64, dtype=torch.bool)
    bad[0, 0, 50] = bad[1, 1, 3] = bad[1, 1, 19] = True  # 50 is not rotated, 3 with 19
    assert torch.equal(~torch.isfinite(out).cpu(), bad)
    ref.within(out.cpu()[~bad], want[~bad], bound[~bad], ref.u_of(BF16), "finite")
    out, _ = la.qk_norm_rope(x, None)  # neither norm nor rotation: a copy
    assert torch.equal(torch.isnan(out), torch.isnan(x))  # (a NaN's payload is not kept)
    assert torch.equal(out[~torch.isnan(x)], x[~torch.isnan(x)])
    # rows of zeros: zero, and a zero gradient direction of r only
    z = torch.zeros_like(q)
    out, _ = la.qk_norm_rope(z, None, near, table, q_weight=w[0], eps=1e-6)
    assert (out == 0).all()
    # no tokens: empty outputs, zero weight gradients
    e = q[:0]
    out, _ = la.qk_norm_rope(e, None, near[:0], table, q_weight=w[0])
    assert out.shape == (0, 2, 64)
    _, _, dw, _ = la.qk_norm_rope_backward(e, None, near[:0], table, e, None, q_weight=w[0])
    assert (dw == 0).all()
    with pytest.raises(ValueError):
        la.qk_norm_rope(q.transpose(0, 1), None, None, None)
    with pytest.raises(ValueError):
        la.qk_norm_rope(q, k, near[:3], table)
    with pytest.raises(TypeError):
        la.qk_norm_rope(q.half(), None)
    with pytest.raises(la.LightningAttnError):
        la.qk_norm_rope(q, k, near, table, q_weight=w[0])
    with pytest.raises(la.LightningAttnError):
        la.qk_norm_rope(q[:1].expand(4, 2, 64), None)  # a broadcast input has no row stride


# --------------------------------------------------------------- append
@pytest.mark.parametrize("dtype, t, h, hk, d, page, rot", [
    (BF16, 1, 64, 8, 128, 64, 64), (BF16, 77, 6, 2, 64, 16, 64), (BF16, 50, 3, 3, 128, 1, 128),
    (FP32, 33, 8, 1, 128, 48, 128), (FP32, 5, 2, 2, 64, 7, 16), (BF16, 900, 16, 4, 128, 256, 64)])
def test_paged_append(dtype, t, h, hk, d, page, rot):
    g = gen(6)
    q, k, v = qkv(t, h, hk, d, dtype, g)
    qw, kw = weights(d, g)
    table, pos = la.rotary_table(4096, rot, device="cuda"), positions_of(t, 4096, g)
    pages = -(-(t + 9) // page) + 1
    both = randn((pages, 2, hk, page, d), dtype, g)  # one array of pages, keys and values
    kc, vc = both[:, 0], both[:, 1]
    before = both.clone()
    v.view(torch.int16 if dtype == BF16 else torch.int32)[0, 0, :3] = -5  # NaNs with a payload
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:t].int()
    if t > 4:  # padding and a slot outside the pool: no row written
        slots[1], slots[3] = -1, pages * page
    args = dict(q_weight=qw, k_weight=kw, eps=EPS)
    qo = la.paged_append(q, k, v, pos, table, kc, vc, slots, **args)
    wq, wk = la.qk_norm_rope(q, k, pos, table, **args)
    want, bound = ref.norm_rope(c(k), c(kw), EPS, c(table), c(pos), False)
    ref.within(wk, want, bound, ref.u_of(dtype), "k")
    assert torch.equal(qo, wq)
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            before[s // page, 0, :, s % page] = wk[i]
            before[s // page, 1, :, s % page] = v[i]
    bits = torch.int16 if dtype == BF16 else torch.int32  # values are copied bit for bit
    assert torch.equal(both.view(bits), before.view(bits))


def test_paged_append_no_tokens_and_refusals():
    g = gen(7)
    q, k, v = qkv(3, 4, 2, 64, BF16, g)
    kc = randn((4, 2, 16, 64), BF16, g)
    slots = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    before = kc.clone()
    out = la.paged_append(q[:0], k[:0], v[:0], None, None, kc, kc.clone(), slots[:0])
    assert out.shape == (0, 4, 64) and torch.equal(kc, before)
    for bad in (dict(slots=slots.long()), dict(slots=slots[:2]), dict(v=v[:, :1]), dict(kc=kc[:, :1]),
                dict(kc=kc.float()), dict(kc=kc.transpose(1, 2)), dict(q=q.cpu())):
        a = {**dict(q=q, k=k, v=v, kc=kc, slots=slots), **bad}
        with pytest.raises((ValueError, la.LightningAttnError)):
            la.paged_append(a["q"], a["k"], a["v"], None, None, a["kc"], kc.clone(), a["slots"])
    with pytest.raises(ValueError):
        la.paged_append(q, k, v, slots, None, kc, kc.clone(), slots)  # positions without a table
    # queries rotated in place
    table, pos = la.rotary_table(64, 64, device="cuda"), positions_of(3, 64, g)
    want = la.paged_append(q, k, v, pos, table, kc, kc.clone(), slots)
    assert la.paged_append(q, k, v, pos, table, kc, kc.clone(), slots, q_out=q).data_ptr() == q.data_ptr()
    assert torch.equal(q, want)


# --------------------------------------------------------------- attention
def pool(lens, page, hk, d, dtype, g, spare=2, garbage=float("nan")):
    """Pages of the requests in random places; everything else is garbage."""
    blocks = [-(-n // page) for n in lens]
    pages = sum(blocks) + spare
    order = torch.randperm(pages, generator=g, device="cuda").int()
    bt = torch.full((len(lens), max(max(blocks), 1) + 1), -1, dtype=torch.int32, device="cuda")
    kc = torch.full((pages, hk, page, d), garbage, dtype=dtype, device="cuda")
    vc = kc.clone()
    at = 0
    for i, n in enumerate(lens):
        bt[i, :blocks[i]] = order[at:at + blocks[i]]
        at += blocks[i]
        for cache in (kc, vc):
            x = randn((n, hk, d), dtype, g)
            t = torch.arange(n, device="cuda")
            cache[bt[i, t // page].long(), :, t % page] = x
    return kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda")


def check_attention(q, kc, vc, bt, lens, scale=None, **kw):
    b, h, d = q.shape
    lse = torch.empty((b, h), device="cuda")
    out = la.paged_decode(q, kc, vc, bt, lens, scale=scale, lse=lse, **kw)
    scale = d ** -0.5 if scale is None else scale
    want, wlse, bound, lbound = ref.attention(c(q), c(kc), c(vc), c(bt), c(lens), scale)
    ref.within(out, want, bound, ref.u_of(q.dtype), "out")
    ref.within(lse, wlse, lbound, ref.u_of(FP32), "lse")
    return out


EDGES = [0, 1, 15, 16, 17, 47, 48, 49, 63, 64, 65, 127, 129, 500, 0, 1, 1023]


@pytest.mark.parametrize("page", [1, 5, 16, 48, 64, 256])
@pytest.mark.parametrize("dtype, h, hk, d", [(BF16, 16, 2, 128), (FP32, 6, 2, 64)])
def test_paged_decode_lengths_and_pages(dtype, h, hk, d, page):
    g = gen(page)
    kc, vc, bt, lens = pool(EDGES, page, hk, d, dtype, g)
    check_attention(randn((len(EDGES), h, d), dtype, g), kc, vc, bt, lens)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h, hk", [(1, 1), (4, 4), (3, 1), (8, 1), (9, 1), (16, 1), (40, 2), (64, 8)])
def test_paged_decode_heads(dtype, d, h, hk):
    g = gen(h * d)
    kc, vc, bt, lens = pool([300, 7, 64], 32, hk, d, dtype, g)
    check_attention(randn((3, h, d), dtype, g), kc, vc, bt, lens)


@pytest.mark.parametrize("dtype, lens", [
    (BF16, [40000]), (FP32, [20011]), (BF16, [9000, 3, 0, 17001]), (BF16, [1] * 700),
    (FP32, [130] * 200), (BF16, [0, 0, 0])])
def test_paged_decode_split(dtype, lens):
    """One long request, ragged ones, more units than CTAs, none at all."""
    g = gen(len(lens))
    kc, vc, bt, sl = pool(lens, 64, 2, 64, dtype, g)
    check_attention(randn((len(lens), 8, 64), dtype, g), kc, vc, bt, sl)


@pytest.mark.parametrize("dtype, h, hk, d", [(BF16, 16, 2, 128), (BF16, 12, 1, 64), (FP32, 8, 4, 64),
                                             (FP32, 16, 1, 128)])
@pytest.mark.parametrize("longest", [50, 128, 500, 1900, 4096])
def test_paged_decode_wide_and_narrow_tables(dtype, h, hk, d, longest):
    """The same requests with a table that just holds them (one cluster a unit, of 1
    to 8 CTAs) and one for contexts of 64K tokens (the split over all CTAs)."""
    g = gen(longest + d)
    lens_list = [longest, 0, longest // 3 + 1, 1]
    kc, vc, bt, lens = pool(lens_list, 32, hk, d, dtype, g)
    q = randn((4, h, d), dtype, g)
    bt = bt[:, :-1] if bt.shape[1] > 1 else bt
    check_attention(q, kc, vc, bt, lens)
    wide = torch.full((4, 2048), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.shape[1]] = bt
    check_attention(q, kc, vc, wide, lens)


def test_paged_decode_large_scores():
    """Scores in the hundreds that rise along the cache: the running maximum
    rescales often, and weights underflow."""
    g = gen(11)
    kc, vc, bt, lens = pool([2000, 333], 16, 1, 128, BF16, g)
    ramp = torch.linspace(0.1, 12, kc.shape[2], device="cuda")[None, None, :, None]
    kc = (kc.float() * ramp).to(BF16)
    check_attention(randn((2, 4, 128), BF16, g) * 3, kc, vc, bt, lens, scale=0.7)
    check_attention(randn((2, 4, 128), BF16, g), kc, vc, bt, lens, scale=-0.5)


def test_paged_decode_absent_pages_and_clamped_lengths():
    g = gen(12)
    kc, vc, bt, lens = pool([100, 40, 64], 16, 2, 128, BF16, g)
    bt[0, 2] = -1                 # tokens 32..47 are left out
    bt[1, :3] = 10 ** 9           # none is left
    lens[2] = 2 ** 31 - 1         # more than the table row holds
    bt[2] = bt[0, 0]
    bt[2, -1] = bt[0, 1]
    out = check_attention(randn((3, 4, 128), BF16, g), kc, vc, bt, lens)
    assert (out[1] == 0).all()
    lens[0] = -7
    assert (check_attention(randn((3, 4, 128), BF16, g), kc, vc, bt, lens)[0] == 0).all()


def test_paged_decode_strides_and_guards():
    """Queries as a slice, keys and values as halves of one array, a wider
    table, and an output inside guard rows."""
    g = gen(13)
    kc, vc, bt, lens = pool([65, 200, 9], 16, 2, 64, BF16, g)
    both = torch.stack([kc, vc], dim=1)
    wide = torch.full((3, bt.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.shape[1]] = bt
    x = randn((3, 12, 64), BF16, g)
    buf = torch.full((5, 8, 64), 3.0, dtype=BF16, device="cuda")
    out = check_attention(x[:, :8], both[:, 0], both[:, 1], wide[:, :bt.shape[1]], lens, out=buf[1:4])
    assert (buf[0] == 3).all() and (buf[4] == 3).all() and out.data_ptr() == buf[1].data_ptr()
    assert torch.equal(out, la.paged_decode(x[:, :8].contiguous(), kc, vc, bt, lens))


def test_paged_decode_offsets_past_32_bits():
    """A cache of more than 2^31 elements (and 2^32 bytes) per half, its last pages used."""
    page, hk, d = 64, 8, 128
    pages = 2 ** 31 // (page * hk * d) + 40
    kc = torch.empty((pages, hk, page, d), dtype=BF16, device="cuda")
    vc = torch.empty_like(kc)
    g = gen(14)
    for cache in (kc, vc):
        cache[-12:] = randn((12, hk, page, d), BF16, g)
    bt = torch.arange(pages - 12, pages, device="cuda").int()[None].repeat(2, 1)
    lens = torch.tensor([700, 750], dtype=torch.int32, device="cuda")
    q, k, v = qkv(2, 64, hk, d, BF16, g)
    slots = torch.tensor([(pages - 1) * page + 5, pages * page - 1], dtype=torch.int32, device="cuda")
    q = la.paged_append(q, k, v, None, None, kc, vc, slots)
    out = la.paged_decode(q, kc, vc, bt, lens)
    small = bt - (pages - 12)
    assert torch.equal(kc[-1, :, -1], k[1]) and torch.equal(vc[-1, :, 5], v[0])
    want, _, bound, _ = ref.attention(c(q), c(kc[-12:]), c(vc[-12:]), c(small), c(lens), d ** -0.5)
    ref.within(out, want, bound, ref.u_of(BF16), "out")


@pytest.mark.parametrize("seed", range(24))
def test_paged_decode_random(seed):
    """Seeded random shapes, lengths, pages, strides and garbage."""
    import random
    rng = random.Random(seed)
    dtype, d = rng.choice([BF16, BF16, FP32]), rng.choice([64, 128])
    hk = rng.choice([1, 2, 3, 8])
    h = hk * rng.choice([1, 2, 5, 8, 11, 16])
    page = rng.choice([1, 3, 16, 24, 64, 300])
    b = rng.choice([1, 2, 9, 40])
    most = rng.choice([1, 20, 200, 3000 if b < 20 else 400])
    lens_list = [rng.choice([0, 1, most, rng.randint(0, most)]) for _ in range(b)]
    g = gen(seed)
    kc, vc, bt, lens = pool(lens_list, page, hk, d, dtype, g, garbage=rng.choice([float("nan"),
                                                                             float("-inf"), 3e38]))
    if rng.random() < 0.5:  # a table for longer contexts
        wide = torch.full((b, 20000 // page + bt.shape[1]), -1, dtype=torch.int32, device="cuda")
        wide[:, :bt.shape[1]] = bt
        bt = wide
    x = randn((b, h + rng.choice([0, 2]), d), dtype, g) * rng.choice([0.1, 1, 4])
    x = x.to(dtype)
    check_attention(x[:, :h], kc, vc, bt, lens, scale=rng.choice([None, 0.02, 1.0]))


def test_paged_decode_refusals():
    g = gen(15)
    kc, vc, bt, lens = pool([10, 20], 16, 2, 64, BF16, g)
    q = randn((2, 4, 64), BF16, g)
    for bad in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[:1]), dict(bt=bt.long()),
                dict(lens=lens.long()), dict(lens=lens[:1]), dict(kc=kc.transpose(1, 2)),
                dict(vc=vc[:1]), dict(q=q.transpose(0, 1)), dict(lens=lens.cpu())):
        a = {**dict(q=q, kc=kc, vc=vc, bt=bt, lens=lens), **bad}
        with pytest.raises((ValueError, la.LightningAttnError)):
            la.paged_decode(a["q"], a["kc"], a["vc"], a["bt"], a["lens"])
    with pytest.raises(la.LightningAttnError):
        la.paged_decode(q, kc, vc, bt, lens, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        la.paged_decode(q, kc, vc, bt, lens, lse=torch.empty(2, 4))
    e = la.paged_decode(q[:0], kc, vc, bt[:0], lens[:0])
    assert e.shape == (0, 4, 64)


# -------------------------------------------------------------------- step
@pytest.mark.parametrize("dtype, h, hk, d, rot, inter", [
    (BF16, 64, 8, 128, 64, False), (BF16, 12, 1, 64, 64, True), (FP32, 6, 2, 128, 128, False)])
def test_paged_step(dtype, h, hk, d, rot, inter):
    g = gen(16)
    lens_list = [1, 300, 17, 64, 2000]
    kc, vc, bt, lens = pool(lens_list, 16, hk, d, dtype, g, garbage=float("inf"))
    q, k, v = qkv(5, h, hk, d, dtype, g)
    qw, kw = weights(d, g)
    table = la.rotary_table(4096, rot, device="cuda")
    pos = lens - 1
    slots = bt[torch.arange(5, device="cuda"), (pos // 16).long()] * 16 + pos % 16
    args = dict(q_weight=qw, k_weight=kw, eps=EPS, interleaved=inter)
    lse = torch.empty((5, h), device="cuda")
    k2, v2 = kc.clone(), vc.clone()
    out = la.paged_step(q, k, v, pos, table, kc, vc, slots, bt, lens, lse=lse, **args)
    la.paged_append(q, k, v, pos, table, k2, v2, slots, **args)
    assert torch.equal(kc.view(torch.int16 if dtype == BF16 else torch.int32),
                       k2.view(torch.int16 if dtype == BF16 else torch.int32))
    assert torch.equal(vc.view(torch.int16 if dtype == BF16 else torch.int32),
                       v2.view(torch.int16 if dtype == BF16 else torch.int32))
    rotated, qbound = ref.norm_rope(c(q), c(qw), EPS, c(table), c(pos), inter)
    want, wlse, bound, lbound = ref.attention(rotated, c(kc), c(vc), c(bt), c(lens), d ** -0.5)
    # the queries carry their own fp32 error and (bf16 cache) their split into two
    # bf16 parts, 2^-16 of an element: a score moves by at most that times sum |q k|, which
    # the bound's own score term (2 e (D + 8) of it, 2^-16 at D = 64) already is
    extra = (qbound / rotated.abs().amax(-1, keepdim=True).clamp(min=1e-3)).amax() + 2.0 ** -16
    more = 1 + float(extra) / (2 * ref.E * (d + 8))
    ref.within(out, want, bound * more, ref.u_of(dtype), "out")
    ref.within(lse, wlse, lbound * more, ref.u_of(FP32), "lse")


# ----------------------------------------------------------------- reserve
def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check_reserve(table, lens, new, finished, stack, count, page, num_tokens, in_place):
    bt, sl, fp, fc = ints(table), ints(lens), ints(stack), ints([count])
    done = None if finished is None else torch.tensor(finished, device="cuda")
    out = {} if in_place else dict(seq_lens_out=torch.empty_like(sl), free_count_out=torch.empty_like(fc))
    slots, pos, cu, served = la.paged_reserve(bt, sl, ints(new), fp, fc, page, num_tokens,
                                              finished=done, **out)
    want = ref.reserve(table, lens, new, finished, stack, count, page, num_tokens)
    if not in_place:
        assert sl.tolist() == lens and fc.tolist() == [count]
    assert bt.tolist() == want["table"]
    assert out.get("seq_lens_out", sl).tolist() == want["lens"]
    assert out.get("free_count_out", fc).tolist() == [want["count"]]
    assert fp.tolist() == want["stack"]
    assert slots.tolist() == want["slots"] and pos.tolist() == want["positions"]
    assert cu.tolist() == want["cu"] and served.tolist() == want["served"]
    return want


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("batch, page, pages, longest, new_most, ended, steps", [
    (1, 16, 8, 100, 5, 0.0, 6), (5, 4, 40, 60, 9, 0.3, 12), (128, 64, 700, 600, 1, 0.1, 5),
    (40, 16, 300, 400, 60, 0.2, 8),          # runs out of pages
    (17, 7, 2000, 2000, 900, 0.2, 4),        # over 4096 tokens: eight CTAs
    (2500, 1, 3000, 6, 2, 0.4, 4), (8192, 8, 9000, 40, 3, 0.1, 2)])
def test_paged_reserve_steps(batch, page, pages, longest, new_most, ended, steps, in_place):
    """Several steps of a pool that fills up, tables that overflow, rows that
    end and start again in one step."""
    import random
    rng = random.Random(batch + in_place)
    width = -(-longest // page)
    table, lens = [[-1] * width for _ in range(batch)], [0] * batch
    stack, count = rng.sample(range(pages), pages), pages
    for _ in range(steps):
        new = [rng.randint(-1, new_most) for _ in range(batch)]
        finished = [rng.random() < ended for _ in range(batch)] if ended else None
        total = sum(max(n, 0) for n in new)
        want = check_reserve(table, lens, new, finished, stack, count, page,
                             max(0, total + rng.choice([0, 13, -3])), in_place)
        table, lens, stack, count = want["table"], want["lens"], want["stack"], want["count"]
        held = [p for b in range(batch) for p in table[b][:-(-lens[b] // page)]]
        assert sorted(held + stack[:count]) == list(range(pages))  # no page lost or given twice


def test_paged_reserve_edges():
    # no pages at all; a request that needs none is served
    check_reserve([[3], [-1]], [3, 0], [1, 1], None, [0, 0, 0, 0], 0, 4, 2, True)
    # an empty step, and tokens past the outputs' size
    check_reserve([[3, -1]], [3], [0], None, [1, 2, 0, 0], 2, 4, 0, True)
    check_reserve([[3, -1]], [3], [4], None, [1, 2, 0, 0], 2, 4, 2, True)
    bt, one = ints([[0, 1]]), ints([0])
    for bad in (dict(a=bt.long()), dict(b=ints([1, 2])), dict(p=0)):
        with pytest.raises((ValueError, la.LightningAttnError)):
            la.paged_reserve(bad.get("a", bt), bad.get("b", one), one, ints([0, 1]), one,
                             bad.get("p", 4), 1)
    with pytest.raises(la.LightningAttnError, match="8192"):
        n = 8193
        la.paged_reserve(torch.zeros((n, 1), dtype=torch.int32, device="cuda"), ints([0] * n),
                         ints([0] * n), ints([0]), one, 4, 1)


# ----------------------------------------------------- together, as used
def test_serving_loop_replayed_from_a_graph():
    """Prompts enter through reserve and append, then a captured step (reserve,
    paged_step) is replayed: every output is the dense attention's over what has been
    cached, for requests that end and start on the way."""
    g = gen(20)
    b, h, hk, d, page, pages = 6, 8, 2, 64, 8, 64
    dtype = BF16
    qw, kw = weights(d, g)
    table = la.rotary_table(512, 32, device="cuda")
    args = dict(q_weight=qw, k_weight=kw, eps=EPS)
    kc = torch.full((pages, hk, page, d), float("nan"), dtype=dtype, device="cuda")
    vc = kc.clone()
    bt = torch.full((b, 12), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(b, dtype=torch.int32, device="cuda")
    stack, count = torch.arange(pages, device="cuda").int(), ints([pages])
    seen = [[] for _ in range(b)]  # (k, v) rows of each request, as cached

    def cached(i):
        return ref.gather(c(kc), c(bt[i]), int(lens[i]))[0], ref.gather(c(vc), c(bt[i]), int(lens[i]))[0]

    prompts = [13, 1, 40, 8, 0, 25]
    t = sum(prompts)
    q, k, v = qkv(t + 3, h, hk, d, dtype, g)  # a padded batch
    slots, pos, cu, served = la.paged_reserve(bt, lens, ints(prompts), stack, count, page, t + 3)
    la.paged_append(q, k, v, pos, table, kc, vc, slots, **args)
    _, kr = la.qk_norm_rope(q, k, pos, table, **args)
    assert served.all() and cu[-1] == t and (slots[t:] == -1).all()
    for i in range(b):
        for j in range(int(cu[i]), int(cu[i + 1])):
            seen[i].append((kr[j].cpu().double(), v[j].cpu().double()))
        assert torch.equal(cached(i)[0], torch.stack([x[0] for x in seen[i]])
                           if seen[i] else torch.zeros(0, hk, d, dtype=torch.float64))

    new, done = torch.ones(b, dtype=torch.int32, device="cuda"), torch.zeros(b, dtype=torch.bool, device="cuda")
    x = torch.zeros((b, h + 2 * hk, d), dtype=dtype, device="cuda")
    q, k, v = x[:, :h], x[:, h:h + hk], x[:, h + hk:]

    def step():
        slots, pos, _, served = la.paged_reserve(bt, lens, new, stack, count, page, b, finished=done)
        return la.paged_step(q, k, v, pos, table, kc, vc, slots, bt, lens, **args), pos, served

    side = torch.cuda.Stream()
    keep = [t.clone() for t in (bt, lens, stack, count, kc, vc)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for t, s in zip((bt, lens, stack, count, kc, vc), keep):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, pos, served = step()
    for n in range(10):
        x.copy_(randn(x.shape, dtype, g))
        ended = [n in (3, 7) and i in (1, 2) for i in range(b)]
        done.copy_(torch.tensor(ended))
        for i in range(b):
            if ended[i]:
                seen[i] = []
        graph.replay()
        assert served.all()
        qr, kr = la.qk_norm_rope(q, k, pos, table, **args)
        for i in range(b):
            seen[i].append((kr[i].cpu().double(), v[i].cpu().double()))
            kk, vv = (torch.stack([y[j] for y in seen[i]]) for j in (0, 1))
            assert int(lens[i]) == len(seen[i]) == int(pos[i]) + 1
            rk, rv = cached(i)
            assert torch.equal(rk, kk) and torch.equal(rv, vv)
        rotated, _ = ref.norm_rope(c(q), c(qw), EPS, c(table), c(pos), False)
        want, _, bound, _ = ref.attention(rotated, c(kc), c(vc), c(bt), c(lens), d ** -0.5)
        # as in test_paged_step: the queries' own error beside the scores'
        ref.within(out, want, 4 * bound, ref.u_of(dtype), f"step {n}")


def test_training_pass_through_the_lightning_layer():
    """qk_norm_rope, prefill, backward and qk_norm_rope_backward in a row: the fp32
    gradients are the slopes of the 64-bit chain."""
    g = gen(21)
    h, d, lens = 2, 64, [50, 14]
    t = sum(lens)
    cu = wl.cu_from_lengths(lens).cuda()
    decay = wl.decay_schedule(h).cuda()
    x = randn((t, 3 * h, d), FP32, g)
    q, k, v = x[:, :h], x[:, h:2 * h], x[:, 2 * h:].contiguous()
    qw, kw = [w * d ** -0.5 for w in weights(d, g)]
    table = la.rotary_table(64, 64, device="cuda")
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    args = dict(q_weight=qw, k_weight=kw, eps=EPS)
    dout = randn((t, h, d), FP32, g)

    qr, kr = la.qk_norm_rope(q, k, pos, table, **args)
    la.prefill(qr, kr, v, decay, cu)
    dqr, dkr, dv = la.backward(qr, kr, v, decay, cu, dout)
    dq, dk, dqw, dkw = la.qk_norm_rope_backward(q, k, pos, table, dqr, dkr, **args)

    def loss(q, k, qw, kw):
        a = ref.norm_rope(q, qw, EPS, c(table), c(pos), False)[0]
        b = ref.norm_rope(k, kw, EPS, c(table), c(pos), False)[0]
        o, _ = oracle.recurrent(a.numpy(), b.numpy(), v.cpu().double().numpy(), decay.cpu(), cu.cpu())
        return float((torch.from_numpy(o) * c(dout).double()).sum())

    base = [c(z).double().contiguous() for z in (q, k, qw, kw)]
    cpu, step = torch.Generator().manual_seed(2), 1e-5
    for at, grad in enumerate((dq, dk, dqw, dkw)):
        way = torch.randn(base[at].shape, generator=cpu, dtype=torch.float64)
        ends = []
        for s in (step, -step):
            moved = list(base)
            moved[at] = base[at] + s * way
            ends.append(loss(*moved))
        slope = (ends[0] - ends[1]) / (2 * step)
        got = c(grad).double()
        # the library's fp32 bound for prefill and backward (1e-4 of the RMS an element),
        # with the elements' errors added up without cancelling
        room = 2e-4 * float(got.pow(2).mean().sqrt() * way.abs().sum())
        assert abs(slope - float((got * way).sum())) <= room


@pytest.mark.parametrize("lengths", [(3000, 1700), (30000, 17000)])  # clusters; split and join
def test_two_graphs_and_side_streams(lengths):
    """Two captured steps, each with its own workspace, replayed at once on two
    streams; and calls on a stream that is not the current one."""
    g = gen(22)
    sets = []
    for n in lengths:
        kc, vc, bt, lens = pool([n, 50], 32, 2, 128, BF16, g)
        q = randn((2, 16, 128), BF16, g)
        sets.append((q, kc, vc, bt, lens, la.paged_decode(q, kc, vc, bt, lens)))
    torch.cuda.synchronize()
    graphs = []
    for q, kc, vc, bt, lens, _ in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, la.paged_decode(q, kc, vc, bt, lens)))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, out), s in zip(graphs, sets):
        assert torch.equal(out, s[-1])
    for (q, kc, vc, bt, lens, want), s in zip(sets, streams):
        outs = [la.paged_decode(q, kc, vc, bt, lens, stream=s) for _ in range(4)]
        s.synchronize()
        assert all(torch.equal(o, want) for o in outs)


def test_two_host_threads():
    """Calls from two threads, each on its own stream: results as alone."""
    import threading
    g = gen(24)
    kc, vc, bt, lens = pool([2000, 3, 700], 16, 2, 64, BF16, g)
    wide = torch.full((3, 3000), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.shape[1]] = bt
    q = randn((3, 8, 64), BF16, g)
    case = (FP32, 60, 4, 4, 64, 64, False, True)
    _, x, y, qw, kw, pos, table = norm_inputs(case, 25)
    dy = randn(x.shape, FP32, g)

    def work():
        return (la.paged_decode(q, kc, vc, bt, lens), la.paged_decode(q, kc, vc, wide, lens),
                *la.qk_norm_rope_backward(x, y, pos, table, dy, dy, q_weight=qw, k_weight=kw))

    want = work()
    torch.cuda.synchronize()
    bad = []

    def run():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(30):
                got = work()
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    bad.append(1)

    threads = [threading.Thread(target=run) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_backward_in_a_graph_beside_eager_calls():
    case = (BF16, 130, 8, 2, 128, 64, False, True)
    g, q, k, qw, kw, pos, table = norm_inputs(case, 23)
    dqo, dko = randn(q.shape, BF16, g), randn(k.shape, BF16, g)

    def call():
        return la.qk_norm_rope_backward(q, k, pos, table, dqo, dko, q_weight=qw, k_weight=kw, eps=EPS)

    want = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        graph.replay()
        eager = call()
    torch.cuda.synchronize()
    for a, b, e in zip(want, got, eager):
        assert torch.equal(a, b) and torch.equal(a, e)
