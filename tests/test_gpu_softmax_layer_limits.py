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
