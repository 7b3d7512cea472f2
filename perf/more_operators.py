"""Operators of the softmax layers of a hybrid lightning-attention model that make long and
shared contexts cheap: the bounds of every cache page's keys, the choice of a query's pages by
those bounds, attention over the chosen pages alone, and attention of a batch whose requests
share a long prefix.

Each case is run in its plain form (elementary torch operations in 32 bits, the scores that
decide a choice in 64) or, where ``own`` is true, through the library's entry points; ``exact``
gives the definition in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp32": 4}
_KEEP = 1  # the first and the last page are always among the chosen


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one serving step of 128 requests: every request's new key enters its page's bounds
        dict(name="bounds_step_128", op="bounds", batch=128, kv_heads=8, dim=128, page=64,
             lo=1024, hi=32768, new_lo=1, new_hi=1, dtype="bf16"),
        # prompts of 500 to 32K tokens behind nothing or an earlier turn: ragged ends, small pages
        dict(name="bounds_prompts_9", op="bounds", batch=9, kv_heads=8, dim=128, page=16,
             lo=0, hi=1001, new_lo=500, new_hi=32768, dtype="bf16"),
        # one chat of 32K tokens: latency
        dict(name="select_1x32k", op="select", batch=1, heads=64, kv_heads=8, dim=128, page=64,
             lo=32768, hi=32768, count=32, dtype="bf16"),
        # a full serving batch, contexts of 1K to 32K
        dict(name="select_128", op="select", batch=128, heads=64, kv_heads=8, dim=128, page=64,
             lo=1024, hi=32768, count=64, dtype="bf16"),
        # a small fp32 model, pages that are no power of two, contexts from a single token on
        dict(name="select_fp32_33", op="select", batch=33, heads=16, kv_heads=4, dim=64, page=48,
             lo=1, hi=20011, count=17, dtype="fp32"),
        # one long document, 4096 of its 128K tokens: latency
        dict(name="sparse_1x128k", op="sparse", batch=1, heads=64, kv_heads=8, dim=128, page=64,
             lo=131072, hi=131072, count=64, dtype="bf16"),
        # a full serving batch, up to 4096 tokens each; the shorter requests have fewer
        dict(name="sparse_128", op="sparse", batch=128, heads=64, kv_heads=8, dim=128, page=64,
             lo=1024, hi=16384, count=64, dtype="bf16"),
        # bounds, choice and attention of one layer's step, 20 requests of an fp32 model
        dict(name="sparse_step_20", op="step", batch=20, heads=16, kv_heads=4, dim=64, page=32,
             lo=1, hi=8192, count=40, dtype="fp32"),
        # four short chats behind one system prompt: latency
        dict(name="prefix_4x2k", op="prefix", batch=4, heads=64, kv_heads=8, dim=128, page=64,
             prefix=2048, lo=1, hi=200, dtype="bf16"),
        # a full serving batch behind a prompt of 8K tokens
        dict(name="prefix_128x8k", op="prefix", batch=128, heads=64, kv_heads=8, dim=128, page=64,
             prefix=8192, lo=1, hi=2048, dtype="bf16"),
        # 32 questions about one document of 64K tokens
        dict(name="prefix_32x64k", op="prefix", batch=32, heads=64, kv_heads=8, dim=128, page=16,
             prefix=65536, lo=1, hi=512, dtype="bf16"),
        # a small fp32 model, odd pages, a prefix that ends inside one, requests without own tokens
        dict(name="prefix_fp32_33", op="prefix", batch=33, heads=16, kv_heads=4, dim=64, page=48,
             prefix=4001, lo=0, hi=777, dtype="fp32"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["bounds", "select", "sparse", "step", "prefix", "prefix"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 48, 64, 128])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 3, 4, 7, 8, 16])
    batch = _spread(rng, 1, 128)
    row = kv * dim * _SIZE[dtype]
    # a cache of at most a quarter of the largest listed case's
    most = max(1, min(131072, (1 << 30) // (2 * batch * row)))
    if op == "bounds":
        hi = _spread(rng, 1, most)
        new_hi = rng.choice([1, _spread(rng, 1, hi)])
        hi -= new_hi
        return dict(op=op, batch=batch, kv_heads=kv, dim=dim, page=page, lo=rng.randint(0, hi),
                    hi=hi, new_lo=rng.randint(0, new_hi), new_hi=new_hi, dtype=dtype)
    c = dict(op=op, batch=batch, heads=heads, kv_heads=kv, dim=dim, page=page, dtype=dtype)
    if op == "prefix":
        # no more products than 32 requests of 64 heads, 128 wide, behind 64K tokens; a
        # sixteenth of that in fp32
        work = (1 << 34) // (16 if dtype == "fp32" else 1)
        prefix = _spread(rng, 1, max(1, min(131072, work // (batch * heads * dim))))
        hi = _spread(rng, 1, min(most, 4096))
        return dict(c, prefix=prefix, lo=rng.randint(0, hi), hi=hi)
    hi = _spread(rng, 1, most)
    # no more chosen tokens than the largest listed case's
    count = _spread(rng, 2, min(128, (1 << 29) // (batch * page * kv * dim)))
    return dict(c, lo=rng.randint(1, hi), hi=hi, count=count)


def _between(lo, hi, n):
    """n whole numbers over [lo, hi], in an order that is neither sorted nor random."""
    if n == 1:
        return [hi]
    return [lo + int(round((hi - lo) * ((i * 0.6180339887498949) % 1.0))) for i in range(n)]


def _blocks(tokens, page):
    return -(-tokens // page)


def _lens(c):
    return _between(c["lo"], c["hi"], c["batch"])


def _new(c):
    return _between(c["new_lo"], c["new_hi"], c["batch"])


def _chosen_tokens(c, n):
    """Tokens of a request of n that a choice of pages with its last one among them holds."""
    blocks = _blocks(n, c["page"])
    return min(blocks, c["count"]) * c["page"] - (blocks * c["page"] - n)


def work(c):
    op, size, d, page, kv = c["op"], _SIZE[c["dtype"]], c["dim"], c["page"], c["kv_heads"]
    batch, lens = c["batch"], _lens(c)
    row = kv * d * size           # the keys of a token, half of a page's bounds
    byts, flops = 0, 0
    if op == "bounds":
        new = _new(c)
        touched = sum(_blocks(n + m, page) - n // page for n, m in zip(lens, new) if m)
        begun = sum(1 for n, m in zip(lens, new) if m and n % page)
        # new keys, bounds written, bounds of pages that had tokens, their table entries, lengths
        byts = (sum(new) + 2 * touched + 2 * begun) * row + 4 * touched + 8 * batch
        return {"bytes": byts, "flops": 2 * sum(new) * kv * d}
    if op == "step":              # a page's bounds written a request (the rest is read anyway)
        byts += 2 * batch * row + 4 * batch
    if op in ("select", "step"):
        blocks = sum(_blocks(n, page) for n in lens)
        byts += 2 * blocks * row + 4 * blocks + 4 * batch * kv * c["count"]
        flops += 2 * blocks * c["heads"] * d
        if op == "select":
            return {"bytes": byts + batch * c["heads"] * d * size + 4 * batch, "flops": flops}
    # attention: queries, outputs, lengths
    byts += 2 * batch * c["heads"] * d * size + 4 * batch
    if op == "prefix":
        byts += 2 * (c["prefix"] + sum(lens)) * row
        byts += 4 * (_blocks(c["prefix"], page) + sum(_blocks(n, page) for n in lens))
        return {"bytes": byts, "flops": 4 * (batch * c["prefix"] + sum(lens)) * c["heads"] * d}
    tokens = sum(_chosen_tokens(c, n) for n in lens)
    byts += 2 * tokens * row
    if op == "sparse":            # the choice, a table entry for each chosen page
        byts += 8 * kv * sum(min(_blocks(n, page), c["count"]) for n in lens)
    return {"bytes": byts, "flops": flops + 4 * tokens * c["heads"] * d}


# ------------------------------------------------------------------ inputs
def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(s, blocks, g, spare=3):
    """Tables of rows with blocks[i] pages each, anywhere in a pool; returns its size."""
    need = sum(blocks)
    order = torch.randperm(need + spare, generator=g, device="cuda").int()
    table = torch.full((len(blocks), max(1, max(blocks))), -1, dtype=torch.int32)
    at = torch.arange(table.shape[1])[None] < torch.tensor(blocks)[:, None]
    s["block_table"] = table.cuda()
    s["block_table"][at.cuda()] = order[:need]
    return need + spare


def _normal(shape, c, g):
    return torch.empty(shape, dtype=_DT[c["dtype"]], device="cuda").normal_(generator=g)


def _some_bounds(pages, c, g):
    """Bounds as a page's keys have them: a centre per channel, and what lies around it."""
    mid = torch.empty((pages, c["kv_heads"], c["dim"]), device="cuda").normal_(generator=g)
    reach = torch.empty_like(mid).uniform_(0.5, 2.5, generator=g)
    both = torch.stack([mid.mul_(0.5) - reach, mid + reach], dim=2)
    return both.to(_DT[c["dtype"]])


def _some_choice(c, lens, g):
    """Distinct pages of every request and key-value head, ascending, the last one among them."""
    width = max(_blocks(n, c["page"]) for n in lens)
    blocks = _ints([_blocks(n, c["page"]) for n in lens])[:, None, None]
    x = torch.rand((c["batch"], c["kv_heads"], max(width, c["count"])), generator=g, device="cuda")
    column = torch.arange(x.shape[2], device="cuda")[None, None]
    x = torch.where(column < blocks, x, 2.0)
    x = torch.where(column == blocks - 1, -1.0, x)
    got = torch.argsort(x, dim=2)[..., :c["count"]]
    got = torch.where(got < blocks, got, 1 << 30).sort(dim=2).values
    return torch.where(got < blocks, got, -1).int().contiguous()


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)
    s = {"case": c}
    op, page, d, kv = c["op"], c["page"], c["dim"], c["kv_heads"]
    lens = _lens(c)
    new = _new(c) if op == "bounds" else [1 if op == "step" else 0] * len(lens)
    order = torch.randperm(len(lens), generator=g, device="cuda").tolist()
    lens, new = [lens[i] for i in order], [new[i] for i in order]
    if op == "bounds":
        first, lens = lens, [n + m for n, m in zip(lens, new)]
    else:
        first = [n - m for n, m in zip(lens, new)]
    blocks = [_blocks(n, page) for n in lens]
    if op == "prefix":
        blocks.append(_blocks(c["prefix"], page))
    pages = _tables(s, blocks, g)
    if op == "prefix":  # one row of the table is the shared prefix's
        s["prefix_table"] = s["block_table"][-1].clone()
        s["block_table"] = s["block_table"][:-1, :max(1, max(blocks[:-1]))].contiguous()
        s["prefix_len"] = _ints([c["prefix"]])
    s["seq_lens"] = _ints(lens)
    if op in ("bounds", "step"):
        s["first"] = _ints(first)
    if op != "select":
        s["k_cache"] = _normal((pages, kv, page, d), c, g)
    if op in ("bounds", "select", "step"):
        s["bounds"] = _some_bounds(pages, c, g)
    if op == "bounds":
        return s
    s["q"] = _normal((c["batch"], c["heads"], d), c, g).mul_(1.5)
    if op != "select":
        s["v_cache"] = _normal((pages, kv, page, d), c, g)
    if op == "sparse":
        s["selected"] = _some_choice(c, lens, g)
    return s


# ------------------------------------------------------------- plain forms
def _bounds_plain(s):
    """Minimum and maximum of the new keys of every page they touch, joined with what the page had."""
    c, table, bounds = s["case"], s["block_table"], s["bounds"]
    page = c["page"]
    first, last = s["first"].long(), s["seq_lens"].long()
    column = torch.arange(table.shape[1], device=table.device)[None]
    touched = (column >= (first // page)[:, None]) & (column * page < last[:, None])
    touched &= (first < last)[:, None]
    b, block = touched.nonzero(as_tuple=True)
    at = table[b, block].long()
    t = block[:, None] * page + torch.arange(page, device=table.device)[None]
    fresh = ((t >= first[b, None]) & (t < last[b, None]))[:, None, :, None]
    keys = s["k_cache"][at].float()
    lo = torch.where(fresh, keys, math.inf).amin(2)
    hi = torch.where(fresh, keys, -math.inf).amax(2)
    old = bounds[at].float()
    had = (block * page < first[b])[:, None, None]
    lo = torch.where(had, torch.minimum(lo, old[:, :, 0]), lo)
    hi = torch.where(had, torch.maximum(hi, old[:, :, 1]), hi)
    bounds[at] = torch.stack([lo, hi], dim=2).to(bounds.dtype)
    return bounds


def _select_plain(s):
    """The pages with the largest bounds of q . k, ties to the lower index: scores in 64 bits,
    where two that differ in the 30th bit still have an order."""
    c, q, table = s["case"], s["q"], s["block_table"]
    b, h, d = q.shape
    kv, count = c["kv_heads"], c["count"]
    blocks = ((s["seq_lens"].long() + c["page"] - 1) // c["page"])[:, None, None]
    x = s["bounds"][table.clamp(min=0).long()].permute(0, 2, 3, 4, 1).double()  # [b, kv, 2, d, n]
    g = q.reshape(b, kv, h // kv, d).double()
    score = (g.clamp(max=0.0) @ x[:, :, 0] + g.clamp(min=0.0) @ x[:, :, 1]).amax(2)
    del x
    column = torch.arange(table.shape[1], device=q.device)[None, None]
    score = torch.where((column < _KEEP) | (column >= blocks - _KEEP), math.inf, score)
    score = torch.where(column < blocks, score, -math.inf)
    got = torch.sort(score, dim=2, descending=True, stable=True).indices[..., :count]
    got = torch.nn.functional.pad(got, (0, count - got.shape[2]), value=1 << 30)
    got = torch.where(got < blocks, got, 1 << 30).sort(dim=2).values
    return torch.where(got < blocks, got, -1).int()


def _weights(q, k, here):
    """Scores of [.., rows, d] queries over [.., n, d] keys, masked."""
    x = (q.float() @ k.float().transpose(-1, -2)) * q.shape[-1] ** -0.5
    return x.masked_fill(~here, -math.inf)


def _sparse_plain(s, selected):
    c, q, table, lens = s["case"], s["q"], s["block_table"], s["seq_lens"]
    b, h, d = q.shape
    kv, page = c["kv_heads"], c["page"]
    sel = selected.long()
    block = sel.clamp(min=0)
    at = table.long()[torch.arange(b, device=q.device)[:, None, None], block].clamp(min=0)
    head = torch.arange(kv, device=q.device)[None, :, None]
    t = block[..., None] * page + torch.arange(page, device=q.device)
    here = ((t < lens[:, None, None, None]) & (sel >= 0)[..., None]).flatten(2)
    x = _weights(q.reshape(b, kv, h // kv, d), s["k_cache"][at, head].flatten(2, 3), here[:, :, None])
    x = torch.exp(x - x.amax(-1, keepdim=True))
    v = s["v_cache"][at, head].flatten(2, 3).float().masked_fill(~here[..., None], 0.0)
    return ((x @ v) / x.sum(-1, keepdim=True)).reshape(b, h, d).to(q.dtype)


def _rows(cache, pages):
    """The pages of every row of a table as [.., kv, tokens, d]."""
    x = cache[pages.clamp(min=0).long()].transpose(-4, -3)
    return x.flatten(-3, -2).float()


def _prefix_plain(s):
    c, q = s["case"], s["q"]
    b, h, d = q.shape
    kv, g = c["kv_heads"], h // c["kv_heads"]
    rows = q.reshape(b, kv, g, d)
    both = rows.transpose(0, 1).reshape(kv, b * g, d)
    kp, vp = _rows(s["k_cache"], s["prefix_table"]), _rows(s["v_cache"], s["prefix_table"])
    there = torch.arange(kp.shape[-2], device=q.device) < s["prefix_len"]
    x = _weights(both, kp, there)
    ks, vs = _rows(s["k_cache"], s["block_table"]), _rows(s["v_cache"], s["block_table"])
    here = (torch.arange(ks.shape[-2], device=q.device)[None] < s["seq_lens"][:, None])[:, None, None]
    y = _weights(rows, ks, here)
    x = x.reshape(kv, b, g, -1)
    m = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True).transpose(0, 1))
    x, y = torch.exp(x - m), torch.exp(y - m.transpose(0, 1))
    total = x.sum(-1, keepdim=True).transpose(0, 1) + y.sum(-1, keepdim=True)
    o = (x.reshape(kv, b * g, -1) @ vp.masked_fill(~there[:, None], 0.0)).reshape(kv, b, g, d)
    o = o.transpose(0, 1) + y @ vs.masked_fill(~here.transpose(2, 3), 0.0)
    return (o / total).reshape(b, h, d).to(q.dtype)


def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "bounds":
        return {"bounds": _bounds_plain(s)}
    if op == "select":
        return {"selected": _select_plain(s)}
    if op == "sparse":
        return {"out": _sparse_plain(s, s["selected"])}
    if op == "prefix":
        return {"out": _prefix_plain(s)}
    bounds = _bounds_plain(s)
    selected = _select_plain(s)
    return {"bounds": bounds, "selected": selected, "out": _sparse_plain(s, selected)}


# ----------------------------------------------------- the library's calls
def _run_own(s, op):
    import lightning_attention_attn_gb300 as la
    c, out = s["case"], {}
    if op in ("bounds", "step"):
        la.paged_bounds(s["k_cache"], s["bounds"], s["block_table"], s["first"], s["seq_lens"])
        out["bounds"] = s["bounds"]
    if op in ("select", "step"):
        out["selected"] = la.paged_select(s["q"], s["bounds"], s["block_table"], s["seq_lens"],
                                          c["page"], c["count"], keep_first=_KEEP, keep_last=_KEEP)
    if op in ("sparse", "step"):
        selected = s["selected"] if op == "sparse" else out["selected"]
        out["out"] = la.paged_sparse_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"],
                                            s["seq_lens"], selected)
    if op == "prefix":
        out["out"] = la.paged_prefix_decode(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"],
                                            s["prefix_len"], s["block_table"], s["seq_lens"])
    return out


# -------------------------------------------------------- the definition
def _bounds64(s):
    out = s["bounds"].double()
    page, table = s["case"]["page"], s["block_table"].cpu().tolist()
    k = s["k_cache"]
    for b, (n, m) in enumerate(zip(s["first"].tolist(), s["seq_lens"].tolist())):
        if n >= m:
            continue
        whole = list(range(n // page, _blocks(m, page)))
        begun = whole.pop(0) if n % page else None
        ended = whole.pop() if whole and m % page else None
        if whole:
            at = torch.tensor([table[b][i] for i in whole], device=k.device)
            x = k[at].double()
            out[at] = torch.stack([-(-x).amax(2), x.amax(2)], dim=2)
        for i in (begun, ended):
            if i is not None:
                x = k[table[b][i], :, max(n - i * page, 0):m - i * page].double()
                lo, hi = -(-x).amax(1), x.amax(1)
                if i == begun:
                    old = out[table[b][i]]
                    lo, hi = -torch.maximum(-lo, -old[:, 0]), torch.maximum(hi, old[:, 1])
                out[table[b][i]] = torch.stack([lo, hi], dim=1)
    return out


def _select64(s, bounds):
    """Page by page the largest q_d k_d that its bounds allow, summed over the channels."""
    c, q = s["case"], s["q"].double()
    kv, g = c["kv_heads"], q.shape[1] // c["kv_heads"]
    out = torch.full((q.shape[0], kv, c["count"]), -1, dtype=torch.int32, device=q.device)
    for b, n in enumerate(s["seq_lens"].tolist()):
        blocks = _blocks(n, c["page"])
        x = bounds[s["block_table"][b, :blocks].long()].double().transpose(0, 1)[:, :, None]
        most = torch.full((kv, blocks), -math.inf, dtype=torch.float64, device=q.device)
        for i in range(g):
            r = q[b].reshape(kv, 1, g, -1)[:, :, i:i + 1]
            most = torch.maximum(most, torch.maximum(r * x[..., 0, :], r * x[..., 1, :]).sum(-1).amax(2))
        order = sorted(range(_KEEP)) + [blocks - 1]
        for j in range(kv):
            row = most[j].tolist()
            free = [i for i in range(blocks) if i not in order]
            free.sort(key=lambda i: (-row[i], i))
            got = [i for i in dict.fromkeys(order) if 0 <= i < blocks]
            got = sorted((got + free)[:c["count"]])
            out[b, j, :len(got)] = _ints(got)
    return out


def _attend64(q, k, v):
    p = torch.softmax(q.double() @ k.double().T / math.sqrt(q.shape[-1]), -1)
    return p @ v.double()


def _sparse64(s, selected):
    c, q = s["case"], s["q"]
    page, kv = c["page"], c["kv_heads"]
    g = q.shape[1] // kv
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for b, n in enumerate(s["seq_lens"].tolist()):
        for j in range(kv):
            block = selected[b, j][selected[b, j] >= 0].long()
            t = (block[:, None] * page + torch.arange(page, device=q.device)).flatten()
            k, v = (x[s["block_table"][b, block].long(), j].flatten(0, 1)[t < n]
                    for x in (s["k_cache"], s["v_cache"]))
            out[b, j * g:(j + 1) * g] = _attend64(q[b, j * g:(j + 1) * g], k, v)
    return out


def _prefix64(s):
    c, q = s["case"], s["q"]
    page, kv = c["page"], c["kv_heads"]
    g = q.shape[1] // kv
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    front = s["prefix_table"][:_blocks(c["prefix"], page)].long()
    for j in range(kv):
        kp, vp = (x[front, j].flatten(0, 1)[:c["prefix"]].double()
                  for x in (s["k_cache"], s["v_cache"]))
        for b, n in enumerate(s["seq_lens"].tolist()):
            own_pages = s["block_table"][b, :_blocks(n, page)].long()
            k, v = (x[own_pages, j].flatten(0, 1)[:n].double() for x in (s["k_cache"], s["v_cache"]))
            head = slice(j * g, (j + 1) * g)
            out[b, head] = _attend64(q[b, head], torch.cat([kp, k]), torch.cat([vp, v]))
    return out


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "bounds":
        return {"bounds": _bounds64(s)}
    if op == "select":
        return {"selected": _select64(s, s["bounds"])}
    if op == "sparse":
        return {"out": _sparse64(s, s["selected"])}
    if op == "prefix":
        return {"out": _prefix64(s)}
    bounds = _bounds64(s)
    selected = _select64(s, bounds)
    return {"bounds": bounds, "selected": selected, "out": _sparse64(s, selected)}
