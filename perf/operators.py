"""Operators of the softmax layers that a hybrid lightning-attention model keeps beside its
lightning layers: per-head norms with the position rotation (training, forward and backward),
the same with the write into a paged key-value cache, attention of one new token over that
cache, and the page bookkeeping of a serving step.

Each case is run in its plain form (elementary torch operations in 32 bits) or, where ``own``
is true, through the library's entry points; ``exact`` gives the definition in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp32": 4}
_EPS = 1e-6
_MAX_POSITION = 1 << 18


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one serving step of 128 requests: a token each, some requests just ended
        dict(name="reserve_step_128", op="reserve", batch=128, page=64, lo=1024, hi=32768,
             new_lo=1, new_hi=1, ended=9),
        # sixteen prompts enter an empty part of the pool: 1K to 32K tokens each, small pages
        dict(name="reserve_prompts_16", op="reserve", batch=16, page=16, lo=0, hi=0,
             new_lo=1024, new_hi=32768, ended=0),
        # the smallest call: one request's token, 64 query and 8 key-value heads
        dict(name="append_1", op="append", tokens=1, heads=64, kv_heads=8, dim=128, rot=64,
             page=64, dtype="bf16", pairs=False),
        # an 8K prompt of the same layer enters the cache
        dict(name="append_8k", op="append", tokens=8192, heads=64, kv_heads=8, dim=128, rot=64,
             page=64, dtype="bf16", pairs=False),
        # training: the queries and keys of an 8K-token layer with 64 heads each
        dict(name="norm_rope_8k", op="forward", tokens=8192, heads=64, kv_heads=64, dim=128,
             rot=128, dtype="bf16", pairs=False),
        # and its gradients
        dict(name="norm_rope_back_8k", op="backward", tokens=8192, heads=64, kv_heads=64,
             dim=128, rot=128, dtype="bf16", pairs=False),
        # a small fp32 model: odd length, uneven heads, neighbouring pairs rotated
        dict(name="norm_rope_back_odd", op="backward", tokens=1021, heads=12, kv_heads=4, dim=64,
             rot=64, dtype="fp32", pairs=True),
        # one short chat: latency
        dict(name="decode_1x300", op="decode", batch=1, heads=64, kv_heads=8, dim=128, page=64,
             lo=300, hi=300, dtype="bf16"),
        # a full serving batch, contexts of 1K to 32K
        dict(name="decode_128", op="decode", batch=128, heads=64, kv_heads=8, dim=128, page=64,
             lo=1024, hi=32768, dtype="bf16"),
        # one long document: the work has to be split over the length
        dict(name="decode_1x128k", op="decode", batch=1, heads=64, kv_heads=8, dim=128, page=16,
             lo=131072, hi=131072, dtype="bf16"),
        # a small fp32 model, pages that are no power of two, ragged lengths
        dict(name="decode_fp32_33", op="decode", batch=33, heads=16, kv_heads=4, dim=64, page=48,
             lo=1, hi=4001, dtype="fp32"),
        # a whole serving step of one layer for 20 requests: append, then attention
        dict(name="step_20", op="step", batch=20, heads=64, kv_heads=8, dim=128, rot=64, page=64,
             lo=1, hi=8192, dtype="bf16", pairs=False),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["reserve", "append", "forward", "backward", "decode", "decode", "step"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "reserve":
        batch = _spread(rng, 1, 512)
        hi = _spread(rng, 1, 32768)
        new_hi = rng.choice([1, 1, _spread(rng, 2, 8192)])
        return dict(op=op, batch=batch, page=page, lo=rng.randint(0, hi), hi=hi,
                    new_lo=rng.randint(0, new_hi), new_hi=new_hi, ended=rng.choice([0, 3, 7]))
    kv = rng.choice([1, 2, 4, 8, 16])
    heads = kv * rng.choice([1, 3, 4, 7, 8, 16])
    if op in ("decode", "step"):
        batch = _spread(rng, 1, 128)
        # at most an eighth of the largest listed case's cache
        most = (1 << 30) // (2 * batch * kv * dim * _SIZE[dtype])
        hi = _spread(rng, 1, max(1, min(131072, most)))
        c = dict(op=op, batch=batch, heads=heads, kv_heads=kv, dim=dim, page=page,
                 lo=rng.randint(1, hi), hi=hi, dtype=dtype)
        if op == "step":
            c.update(rot=rng.choice([dim // 2, dim]), pairs=rng.choice([False, True]))
        return c
    c = dict(op=op, tokens=_spread(rng, 1, 4096), heads=heads, kv_heads=kv, dim=dim,
             rot=rng.choice([dim // 2, dim]), dtype=dtype, pairs=rng.choice([False, True]))
    if op == "append":
        c["page"] = page
    return c


def _between(lo, hi, n):
    """n whole numbers over [lo, hi], in an order that is neither sorted nor random."""
    if n == 1:
        return [hi]
    return [lo + int(round((hi - lo) * ((i * 0.6180339887498949) % 1.0))) for i in range(n)]


def _blocks(tokens, page):
    return -(-tokens // page)


def _reserve_sizes(c):
    lens = _between(c["lo"], c["hi"], c["batch"])
    new = _between(c["new_lo"], c["new_hi"], c["batch"])
    ended = [c["ended"] > 0 and i % (c["ended"] + 1) == c["ended"] for i in range(c["batch"])]
    new = [0 if e else n for n, e in zip(new, ended)]
    return lens, new, ended


def work(c):
    op = c["op"]
    if op == "reserve":
        lens, new, ended = _reserve_sizes(c)
        freed = sum(_blocks(n, c["page"]) for n, e in zip(lens, ended) if e)
        taken = sum(_blocks(n + m, c["page"]) - _blocks(n, c["page"])
                    for n, m, e in zip(lens, new, ended) if not e)
        total = sum(new)
        # lengths, new lengths and flags in; lengths, offsets and flags out; freed pages read
        # from the table and pushed, taken ones popped and entered; a slot and a position a token
        byts = c["batch"] * (4 + 4 + 1 + 4 + 4 + 1) + 8 * (freed + taken) + 8 * total
        return {"bytes": byts, "flops": 8 * (c["batch"] + total)}
    size, d = _SIZE[c["dtype"]], c["dim"]
    if op in ("append", "forward", "backward", "step"):
        t = c["tokens"] if "tokens" in c else c["batch"]
        rows = t * (c["heads"] + c["kv_heads"])
        table = t * c["rot"] * 4
        prep = 2 * rows * d * size + table + 4 * t
        flops = rows * (4 * d + 3 * c["rot"])
        if op == "forward":
            return {"bytes": prep, "flops": flops}
        if op == "backward":
            return {"bytes": 3 * rows * d * size + table + 4 * t, "flops": rows * (11 * d + 3 * c["rot"])}
        prep += 2 * t * c["kv_heads"] * d * size + 4 * t
        if op == "append":
            return {"bytes": prep, "flops": flops}
    lens = _between(c["lo"], c["hi"], c["batch"])
    total = sum(lens)
    byts = 2 * total * c["kv_heads"] * d * size + 4 * sum(_blocks(n, c["page"]) for n in lens)
    byts += 2 * c["batch"] * c["heads"] * d * size + 4 * c["batch"]
    fl = 4 * total * c["heads"] * d
    if op == "step":
        # the new keys and values are counted once, as the cache rows that the attention reads;
        # the queries pass from one half to the other
        byts += prep - 2 * c["batch"] * c["heads"] * d * size
        fl += flops
    return {"bytes": byts, "flops": fl}


# ------------------------------------------------------------------ inputs
def _table(rot, device):
    """cos and sin of every position, [positions, rot]: built once by a program, in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(_MAX_POSITION, dtype=torch.float64, device=device)[:, None] * inv[None]
    return torch.cat([a.cos(), a.sin()], dim=1).float()


_tables = {}


def _shared_table(rot):
    # a model's table is one for all layers and all calls
    if rot not in _tables:
        _tables[rot] = _table(rot, "cuda")
    return _tables[rot]


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pool(s, c, g, blocks, spare):
    """A page pool with the requests' pages anywhere in it, and their table."""
    need = sum(blocks)
    pages = need + spare
    order = torch.randperm(pages, generator=g, device="cuda").int()
    width = max(1, max(blocks))
    table = torch.full((len(blocks), width), -1, dtype=torch.int32)
    at = torch.arange(width)[None] < torch.tensor(blocks)[:, None]
    s["block_table"] = table.cuda()
    s["block_table"][at.cuda()] = order[:need]
    return pages, order


def _cache(s, c, g, pages):
    shape = (pages, c["kv_heads"], c["page"], c["dim"])
    for name in ("k_cache", "v_cache"):
        s[name] = torch.empty(shape, dtype=_DT[c["dtype"]], device="cuda").normal_(generator=g)


def _qkv(s, c, g, tokens, with_v):
    """q, k (and v) as slices of one projection's output, and the two norms' weights."""
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    n = h + (2 if with_v else 1) * hk
    x = torch.empty((tokens, n, d), dtype=_DT[c["dtype"]], device="cuda").normal_(generator=g)
    x.mul_(1.5)
    s["q"], s["k"] = x[:, :h], x[:, h:h + hk]
    if with_v:
        s["v"] = x[:, h + hk:]
    for name in ("q_weight", "k_weight"):
        s[name] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
    s["table"] = _shared_table(c["rot"])


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    s = {"case": c}
    op = c["op"]
    if op == "reserve":
        lens, new, ended = _reserve_sizes(c)
        blocks = [_blocks(n, c["page"]) for n in lens]
        grow = sum(_blocks(n + m, c["page"]) - b for n, m, b in zip(lens, new, blocks))
        pages, order = _pool(s, c, g, blocks, spare=grow + 64)
        width = max(_blocks(n + m, c["page"]) for n, m in zip(lens, new)) + 1
        wide = torch.full((c["batch"], width), -1, dtype=torch.int32, device="cuda")
        wide[:, :s["block_table"].shape[1]] = s["block_table"][:, :width]
        s.update(block_table=wide, seq_lens=_ints(lens), new_lens=_ints(new),
                 finished=torch.tensor(ended, device="cuda") if c["ended"] else None,
                 free_pages=torch.full((pages,), -1, dtype=torch.int32, device="cuda"),
                 free_count=_ints([pages - sum(blocks)]), tokens=max(1, sum(new)),
                 lens_out=torch.empty(c["batch"], dtype=torch.int32, device="cuda"),
                 count_out=torch.empty(1, dtype=torch.int32, device="cuda"))
        s["free_pages"][:pages - sum(blocks)] = order[sum(blocks):]
        return s
    if op in ("forward", "backward"):
        t = c["tokens"]
        _qkv(s, c, g, t, False)
        start = int(torch.randint(0, _MAX_POSITION - t, (1,), generator=g, device="cuda"))
        s["positions"] = torch.arange(start, start + t, dtype=torch.int32, device="cuda")
        if op == "backward":
            for name, x in (("dq", s["q"]), ("dk", s["k"])):
                s[name] = torch.empty(x.shape, dtype=x.dtype, device="cuda").normal_(generator=g)
        return s
    if op == "append":
        t = c["tokens"]
        _qkv(s, c, g, t, True)
        pages = _blocks(t, c["page"]) + 1
        _cache(s, c, g, pages)
        order = torch.randperm(pages, generator=g, device="cuda")
        i = torch.arange(t, device="cuda") + c["page"] // 3
        s["slots"] = (order[i // c["page"]] * c["page"] + i % c["page"]).int()
        start = int(torch.randint(0, _MAX_POSITION - t, (1,), generator=g, device="cuda"))
        s["positions"] = torch.arange(start, start + t, dtype=torch.int32, device="cuda")
        return s
    lens = _between(c["lo"], c["hi"], c["batch"])
    lens = [lens[i] for i in torch.randperm(len(lens), generator=g, device="cuda").tolist()]
    pages, _ = _pool(s, c, g, [_blocks(n, c["page"]) for n in lens], spare=3)
    _cache(s, c, g, pages)
    s["seq_lens"] = _ints(lens)
    if op == "step":
        _qkv(s, c, g, c["batch"], True)
        s["positions"] = s["seq_lens"] - 1
        p = s["positions"].long()
        page = s["block_table"].gather(1, (p // c["page"])[:, None])[:, 0]
        s["slots"] = (page * c["page"] + p % c["page"]).int()
    else:
        s["q"] = torch.empty((c["batch"], c["heads"], c["dim"]), dtype=_DT[c["dtype"]],
                             device="cuda").normal_(generator=g)
    return s


# ------------------------------------------------------------- plain forms
def _angles(table, positions):
    a = table[positions.long()]
    r = a.shape[1] // 2
    return a[:, None, :r], a[:, None, r:]


def _rotate(x, cos, sin, pairs):
    r = 2 * cos.shape[-1]
    if pairs:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., r:]], dim=-1)


def _norm_rope(x, w, cos, sin, pairs):
    f = x.float()
    n = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + _EPS) * w
    return _rotate(n, cos, sin, pairs)


def _norm_rope_back(x, w, dy, cos, sin, pairs):
    f = x.float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + _EPS)
    n = f * r
    g = _rotate(dy.float(), cos, -sin, pairs)
    dw = (g * n).sum((0, 1), dtype=torch.float64).float()
    g = g * w
    return (r * (g - n * (g * n).mean(-1, keepdim=True))).to(x.dtype), dw


def _append_plain(s):
    cos, sin = _angles(s["table"], s["positions"])
    pairs, page = s["case"]["pairs"], s["k_cache"].shape[2]
    slots = s["slots"].long()
    at = (slots // page, slice(None), slots % page)
    s["k_cache"][at] = _norm_rope(s["k"], s["k_weight"], cos, sin, pairs).to(s["k"].dtype)
    s["v_cache"][at] = s["v"]
    return _norm_rope(s["q"], s["q_weight"], cos, sin, pairs)


def _gather(cache, block_table):
    b, n = block_table.shape
    _, hk, page, d = cache.shape
    x = cache[block_table.clamp(min=0).long()]
    return x.transpose(1, 2).reshape(b, hk, n * page, d).float()


def _attend_plain(q, s):
    b, h, d = q.shape
    hk, page = s["k_cache"].shape[1:3]
    n = s["block_table"].shape[1] * page
    here = (torch.arange(n, device=q.device)[None] < s["seq_lens"][:, None])[:, None]
    k = _gather(s["k_cache"], s["block_table"])
    x = (q.float().reshape(b, hk, h // hk, d) @ k.transpose(2, 3)) * d ** -0.5
    del k
    x = x.masked_fill(~here[:, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    v = _gather(s["v_cache"], s["block_table"]).masked_fill(~here[..., None], 0.0)
    return ((x @ v) / x.sum(-1, keepdim=True)).reshape(b, h, d).to(s["v_cache"].dtype)


def _reserve_plain(s):
    page, width = s["case"]["page"], s["block_table"].shape[1]
    table, pages = s["block_table"].long(), s["free_pages"].numel()
    column = torch.arange(width, device=table.device)[None]
    old, new, count = s["seq_lens"].long(), s["new_lens"].long(), s["free_count"].long()
    stack = torch.cat([s["free_pages"].long(), s["free_pages"].new_zeros(1).long()])
    if s["finished"] is not None:
        freed = (column < ((old + page - 1) // page)[:, None]) & s["finished"][:, None]
        to = count + torch.cumsum(freed.flatten(), 0) - 1
        stack[torch.where(freed.flatten(), to, pages)] = table.flatten()
        count = count + freed.sum()
        old = torch.where(s["finished"], 0, old)
    have, want = (old + page - 1) // page, (old + new + page - 1) // page
    need = torch.where(want <= width, want - have, 0)
    upto = torch.cumsum(need, 0)
    served = (want <= width) & ((need == 0) | (upto <= count))
    first = count - 1 - (upto - need)
    here = (column >= have[:, None]) & (column < want[:, None]) & served[:, None]
    top = (first[:, None] - (column - have[:, None])).clamp(0, pages)
    table = torch.where(here, stack[top], table)
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    t = torch.arange(s["tokens"], device=table.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=old.numel() - 1)
    position = old[b] + t - cu[b]
    there = (t < cu[-1]) & served[b]
    block = (position // page).clamp(max=width - 1)
    slots = torch.where(there, table[b, block] * page + position % page, -1)
    return {"slots": slots.int(), "positions": torch.where(there, position, 0).int(),
            "cu_seqlens": cu.int(), "served": served, "block_table": table.int(),
            "seq_lens": torch.where(served, old + new, old).int(),
            "free_pages": stack[:pages].int(),
            "free_count": (count - torch.where(served, need, 0).sum()).int()}


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        return _run_own(s, c, op)
    if op == "reserve":
        return _reserve_plain(s)
    if op == "append":
        return {"q": _append_plain(s).to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "decode":
        return {"out": _attend_plain(s["q"], s)}
    if op == "step":
        return {"out": _attend_plain(_append_plain(s), s), "k_cache": s["k_cache"],
                "v_cache": s["v_cache"]}
    cos, sin = _angles(s["table"], s["positions"])
    if op == "forward":
        return {n: _norm_rope(s[n], s[n + "_weight"], cos, sin, c["pairs"]).to(s[n].dtype)
                for n in ("q", "k")}
    dq, dqw = _norm_rope_back(s["q"], s["q_weight"], s["dq"], cos, sin, c["pairs"])
    dk, dkw = _norm_rope_back(s["k"], s["k_weight"], s["dk"], cos, sin, c["pairs"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


# ----------------------------------------------------- the library's calls
def _run_own(s, c, op):
    import lightning_attention_attn_gb300 as la
    if op == "reserve":
        slots, positions, cu, served = la.paged_reserve(
            s["block_table"], s["seq_lens"], s["new_lens"], s["free_pages"], s["free_count"],
            c["page"], s["tokens"], finished=s["finished"], seq_lens_out=s["lens_out"],
            free_count_out=s["count_out"])
        return {"slots": slots, "positions": positions, "cu_seqlens": cu, "served": served,
                "block_table": s["block_table"], "seq_lens": s["lens_out"],
                "free_pages": s["free_pages"], "free_count": s["count_out"]}
    if op == "decode":
        return {"out": la.paged_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"],
                                       s["seq_lens"])}
    norm = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=_EPS,
                interleaved=c["pairs"])
    if op == "append":
        q = la.paged_append(s["q"], s["k"], s["v"], s["positions"], s["table"], s["k_cache"],
                            s["v_cache"], s["slots"], **norm)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "step":
        out = la.paged_step(s["q"], s["k"], s["v"], s["positions"], s["table"], s["k_cache"],
                            s["v_cache"], s["slots"], s["block_table"], s["seq_lens"], **norm)
        return {"out": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "forward":
        q, k = la.qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], **norm)
        return {"q": q, "k": k}
    dq, dk, dqw, dkw = la.qk_norm_rope_backward(s["q"], s["k"], s["positions"], s["table"],
                                                s["dq"], s["dk"], **norm)
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


# -------------------------------------------------------- the definition
def _turn64(x, table, positions, pairs, back=False):
    """Every pair (a, b) as the complex number a + i b times e^(i angle), in 64 bits."""
    r = table.shape[1]
    row = table[positions.long()].double()
    w = torch.complex(row[:, :r // 2], -row[:, r // 2:] if back else row[:, r // 2:])[:, None]
    i = torch.arange(r // 2, device=x.device)
    first, second = (2 * i, 2 * i + 1) if pairs else (i, i + r // 2)
    z = torch.complex(x[..., first], x[..., second]) * w
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _norm64(x, weight):
    x = x.double()
    return x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + _EPS).sqrt() * weight.double()


def _forward64(x, weight, s, pairs):
    return _turn64(_norm64(x, weight), s["table"], s["positions"], pairs)


def _backward64(x, weight, dy, s, pairs):
    g = _turn64(dy.double(), s["table"], s["positions"], pairs, back=True)
    x, w, d = x.double(), weight.double(), x.shape[-1]
    root = ((x ** 2).sum(-1, keepdim=True) / d + _EPS).sqrt()
    dw = torch.einsum("thd,thd->d", g, x / root)
    dot = torch.einsum("thd,thd,d->th", g, x, w)[..., None]
    return g * w / root - x * dot / (d * root ** 3), dw


def _attend64(q, k_cache, v_cache, block_table, lens):
    h, d = q.shape[1:]
    hk, page = k_cache.shape[1:3]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for b, n in enumerate(lens.tolist()):
        pages = block_table[b, :_blocks(n, page)].long()
        for head in range(hk):
            k = k_cache[pages, head].reshape(-1, d)[:n].double()
            v = v_cache[pages, head].reshape(-1, d)[:n].double()
            group = slice(head * (h // hk), (head + 1) * (h // hk))
            p = torch.softmax(q[b, group].double() @ k.T / math.sqrt(d), -1)
            out[b, group] = p @ v
    return out


def _reserve_exact(s):
    page = s["case"]["page"]
    table, stack = s["block_table"].cpu().tolist(), s["free_pages"].cpu().tolist()
    lens, new, count = s["seq_lens"].tolist(), s["new_lens"].tolist(), int(s["free_count"])
    ended = s["finished"].tolist() if s["finished"] is not None else [False] * len(lens)
    for b, e in enumerate(ended):
        if e:
            for i in range(_blocks(lens[b], page)):
                stack[count] = table[b][i]
                count += 1
            lens[b] = 0
    slots, positions, cu, served = [], [], [0], []
    left, asked = count, 0
    for b, n in enumerate(new):
        have, want = _blocks(lens[b], page), _blocks(lens[b] + n, page)
        fits = want <= len(table[b])
        asked += want - have if fits else 0
        ok = fits and (want == have or asked <= left)
        served.append(ok)
        if ok:
            for i in range(have, want):
                count -= 1
                table[b][i] = stack[count]
        for i in range(n):
            p = lens[b] + i
            slots.append(table[b][p // page] * page + p % page if ok else -1)
            positions.append(p if ok else 0)
        lens[b] += n if ok else 0
        cu.append(cu[-1] + n)
    pad = s["tokens"] - len(slots)
    slots, positions = slots + [-1] * pad, positions + [0] * pad
    return {"slots": _ints(slots), "positions": _ints(positions), "cu_seqlens": _ints(cu),
            "served": torch.tensor(served, device="cuda"), "block_table": _ints(table),
            "seq_lens": _ints(lens), "free_pages": _ints(stack), "free_count": _ints([count])}


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "reserve":
        return _reserve_exact(s)
    if op == "decode":
        return {"out": _attend64(s["q"], s["k_cache"], s["v_cache"], s["block_table"],
                                 s["seq_lens"])}
    q = _forward64(s["q"], s["q_weight"], s, c["pairs"]) if op != "backward" else None
    if op == "forward":
        return {"q": q, "k": _forward64(s["k"], s["k_weight"], s, c["pairs"])}
    if op == "backward":
        dq, dqw = _backward64(s["q"], s["q_weight"], s["dq"], s, c["pairs"])
        dk, dkw = _backward64(s["k"], s["k_weight"], s["dk"], s, c["pairs"])
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    k = _forward64(s["k"], s["k_weight"], s, c["pairs"])
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    page = s["k_cache"].shape[2]
    for i, slot in enumerate(s["slots"].tolist()):
        kc[slot // page, :, slot % page] = k[i]
        vc[slot // page, :, slot % page] = s["v"][i].double()
    if op == "append":
        return {"q": q, "k_cache": kc, "v_cache": vc}
    return {"out": _attend64(q, kc, vc, s["block_table"], s["seq_lens"]), "k_cache": kc,
            "v_cache": vc}
