"""64-bit reference of the softmax layers' operators (CPU, torch float64 and
plain Python), and the error bounds of the GPU tests.

Bounds.  u = eps / 2 of the output's type is the rounding of the result (half
a step: 2^-8 for bf16, 2^-24 for fp32); the arithmetic before it is fp32 with
e = 2^-24 per operation.

* norm + rotation: mean of squares (8 products a lane, 5 levels), rsqrt (2
  ulp), two products, one rotation (2 products, 1 sum): under 32 operations, each
  relative to the pair's size, which is at most sqrt(2) max |n| of the row:
      u |y| + 32 e 2 max|n|
* its gradient: dx = r (w g - h mean(w g h)): each of the two terms carries the
  errors of r, of the rotated g and of a D-term sum of which every partial sum is at
  most sum |w g h|:  u |dx| + 64 e r (max|w g| + max|h| mean|w g h|)
* weight gradients over n rows: a lane adds its rows one by one (at most n / 64 beyond
  the first 64, by the grid), then fewer than 64 further levels:
      u |dw| + (128 + n / 64) e sum |g h|
* attention over n tokens: a score is a D-term sum (the tensor core keeps at least
  23 bits: 2 e an addition), times the scale, into exp2 (2 ulp):
      ds = 2 e (D + 8) scale max_t sum |q k| + 8 e;
  the weights are off by ds in numerator and denominator, by 2^-16 where they are split
  into two bf16 parts, and the sums by one rounding per group of 16 tokens a warp, the warps
  and the pieces:  u |out| + (2 ds + 2^-16 + 2 e (n / 16 + 64)) sum p |v|
"""
import math

import torch

E = 2.0 ** -24


def u_of(dtype):
    return torch.finfo(dtype).eps / 2


def rotate(x, table, positions, interleaved, back=False):
    """x [T, H, d] float64; the rotation of every token's position."""
    if table is None:
        return x.clone()
    r = table.shape[1] // 2
    row = table.double()[positions.long().clamp(0, table.shape[0] - 1)]
    c, s = row[:, None, :r], row[:, None, r:]
    s = -s if back else s
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * r:2], x[..., 1:2 * r:2]
        y[..., 0:2 * r:2], y[..., 1:2 * r:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :r], x[..., r:2 * r]
        y[..., :r], y[..., r:2 * r] = a * c - b * s, a * s + b * c
    return y


def norm(x, weight, eps):
    x = x.double()
    if weight is None:
        return x.clone()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()


def norm_rope(x, weight, eps, table, positions, interleaved):
    """The rotated rows and their bound's arithmetic part."""
    n = norm(x, weight, eps)
    return (rotate(n, table, positions, interleaved),
            (64 * E * n.abs().amax(-1, keepdim=True)).expand(n.shape))


def norm_rope_backward(x, weight, eps, table, positions, interleaved, dy):
    """dx, dweight and the arithmetic parts of their bounds."""
    x, g = x.double(), rotate(dy.double(), table, positions, interleaved, back=True)
    if weight is None:
        return g, None, (64 * E * g.abs().amax(-1, keepdim=True)).expand(g.shape), None
    w, d = weight.double(), x.shape[-1]
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    h = x * r
    wg = w * g
    dx = r * (wg - h * (wg * h).mean(-1, keepdim=True))
    bound = 64 * E * r * (wg.abs().amax(-1, keepdim=True) +
                          h.abs().amax(-1, keepdim=True) * (wg * h).abs().mean(-1, keepdim=True))
    rows = x.shape[0] * x.shape[1]
    return (dx, (g * h).sum((0, 1)), bound.expand(dx.shape),
            (128 + rows / 64) * E * (g * h).abs().sum((0, 1)))


def gather(cache, row, n):
    """The first n tokens of a request: [n, Hkv, d] and which are present."""
    page = cache.shape[2]
    t = torch.arange(n)
    p = row[t // page].long()
    ok = (p >= 0) & (p < cache.shape[0])
    return cache[p.clamp(0, max(cache.shape[0] - 1, 0)), :, t % page].double(), ok


def attention(q, k_cache, v_cache, block_table, seq_lens, scale):
    """out, lse [B, H] and the arithmetic parts of their bounds."""
    q = q.double()
    b, h, d = q.shape
    hk, page = k_cache.shape[1], k_cache.shape[2]
    out, bound = torch.zeros(b, h, d, dtype=torch.float64), torch.zeros(b, h, d, dtype=torch.float64)
    lse = torch.full((b, h), -math.inf, dtype=torch.float64)
    lse_bound = torch.zeros(b, h, dtype=torch.float64)
    for i in range(b):
        n = min(max(int(seq_lens[i]), 0), block_table.shape[1] * page)
        k, ok = gather(k_cache, block_table[i], n)
        v, _ = gather(v_cache, block_table[i], n)
        k, v = k[ok], v[ok]
        if not len(k):
            continue
        g = h // hk
        qg = q[i].reshape(hk, g, d)
        s = torch.einsum("jgd,tjd->jgt", qg, k) * scale
        size = torch.einsum("jgd,tjd->jgt", qg.abs(), k.abs()).amax(-1) * abs(scale)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        p = p / l
        out[i] = torch.einsum("jgt,tjd->jgd", p, v).reshape(h, d)
        ds = 2 * E * (d + 8) * size + 8 * E
        factor = 2 * ds + 2.0 ** -16 + 2 * E * (len(k) / 16 + 64)
        bound[i] = (factor[..., None] * torch.einsum("jgt,tjd->jgd", p, v.abs())).reshape(h, d)
        lse[i] = (m + torch.log(l)).reshape(h)
        # the logarithm, its product and sum with the maximum in fp32
        lse_bound[i] = factor.reshape(h) + 4 * E * (lse[i].abs() + m.reshape(h).abs() + 1)
    return out, lse, bound, lse_bound


def reserve(table, lens, new, finished, free_pages, count, page, num_tokens):
    """paged_reserve on plain lists; returns the new values of everything."""
    table, lens, stack = [list(r) for r in table], list(lens), list(free_pages)
    for b in range(len(lens)):
        if finished is not None and finished[b]:
            for i in range(-(-lens[b] // page)):
                stack[count] = table[b][i]
                count += 1
            lens[b] = 0
    slots, positions, cu, served, asked, free = [], [], [0], [], 0, count
    for b, n in enumerate(new):
        n = max(n, 0)
        have, want = -(-lens[b] // page), -(-(lens[b] + n) // page)
        need = want - have if want <= len(table[b]) else 0
        asked += need
        ok = want <= len(table[b]) and (need == 0 or asked <= free)
        served.append(ok)
        if ok:
            for i in range(have, want):
                count -= 1
                table[b][i] = stack[count]
        for t in range(lens[b], lens[b] + n):
            slots.append(table[b][t // page] * page + t % page if ok else -1)
            positions.append(t if ok else 0)
        lens[b] += n if ok else 0
        cu.append(cu[-1] + n)
    slots, positions = slots[:num_tokens], positions[:num_tokens]
    pad = num_tokens - len(slots)
    return dict(table=table, lens=lens, stack=stack, count=count, slots=slots + [-1] * pad,
                positions=positions + [0] * pad, cu=cu, served=served)


def within(got, ref, bound, u, what=""):
    """Every element within bound + u |ref| (and infinities equal)."""
    got, ref = got.detach().cpu().double(), ref.double()
    same = torch.isinf(ref)
    assert torch.equal(got[same], ref[same]), f"{what}: infinities differ"
    err = (got - ref).abs()[~same]
    room = (bound + u * ref.abs())[~same]
    bad = ~(err <= room)
    if err.numel():
        print(f"[{what}] worst err / bound {float((err / room.clamp(min=1e-300)).max()):.3f}")
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} elements off, worst "
                           f"{float((err - room).max()):.3e} beyond its bound")
