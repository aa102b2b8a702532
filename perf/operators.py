"""Attention over a paged key-value cache: what is measured, and on which sizes.

Four operators that a decoder layer needs next to its quantized linears:

  append   rotate the query and key heads of a fused QKV output by their positions and write keys and values
           into the pages of a cache
  decode   attention of one new token per sequence over its pages
  prefill  causal attention of packed prompts with grouped heads, over packed keys ("packed") or over the
           pages of a cache that already holds earlier tokens ("paged")
  pages    bookkeeping of the cache: "fork" gives children their parent's pages, "compact" moves the live
           pages to the front

Shapes: T tokens, Hq query heads, Hkv key-value heads (Hq a multiple), D channels of a head, pages of `page`
tokens; a cache plane is [pages][Hkv][page][D], a table row lists the pages of one sequence in order.

The plain forms below are elementary torch operations in fp32, rounded once.  `exact` states the definitions
again in fp64.
"""

import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
LOWEST = float("-inf")

# (query heads, key-value heads, channels): grouped heads of 4, 7, 8 and 5, plain heads, one shared head,
# narrow heads
HEADS = [(32, 8, 128), (28, 4, 128), (64, 8, 128), (40, 8, 128), (32, 32, 128), (8, 1, 128), (14, 2, 64), (12, 12, 64),
         (71, 1, 64)]
PAGES = [16, 32, 64, 128]


# ----------------------------------------------------------------------------------------------------------
# cases


def _heads(h):
    return {"hq": h[0], "hkv": h[1], "d": h[2]}


def listed():
    g4, g7, g8, narrow = _heads((32, 8, 128)), _heads((28, 4, 128)), _heads((64, 8, 128)), _heads((14, 2, 64))
    return [
        # one decode step of a small batch: each sequence appends one token; a pure latency case
        {"name": "append step", "op": "append", "mode": "step", "seqs": 16, "longest": 4096, **g4, "page": 16, "type": "bf16"},
        # the prompts of a prefill batch, several thousand tokens of ragged sequences at once
        {"name": "append prompts", "op": "append", "mode": "prompt", "seqs": 7, "longest": 2048, **g4, "page": 64, "type": "f16"},
        # a single user's chat: one sequence, a few hundred tokens; latency
        {"name": "decode one short", "op": "decode", "seqs": 1, "longest": 333, **g4, "page": 16, "type": "bf16"},
        # a served batch of ragged contexts, some slots empty
        {"name": "decode batch ragged", "op": "decode", "seqs": 48, "longest": 4096, **g7, "page": 32, "type": "f16"},
        # one very long document: few rows, so the cache's length has to be split
        {"name": "decode one long", "op": "decode", "seqs": 1, "longest": 131072, **g8, "page": 64, "type": "bf16"},
        # long contexts in a batch: the bandwidth case, the largest cache
        {"name": "decode batch long", "op": "decode", "seqs": 16, "longest": 32768, **g4, "page": 128, "type": "bf16"},
        # one short prompt of odd length on a small model's narrow heads
        {"name": "prefill short", "op": "prefill", "mode": "packed", "seqs": 1, "longest": 77, **narrow, "page": 0, "type": "f16"},
        # a batch of ragged prompts
        {"name": "prefill ragged", "op": "prefill", "mode": "packed", "seqs": 9, "longest": 1531, **g4, "page": 0, "type": "bf16"},
        # one long prompt: the compute-bound case
        {"name": "prefill long", "op": "prefill", "mode": "packed", "seqs": 1, "longest": 8192, **g4, "page": 0, "type": "bf16"},
        # chunks of new tokens behind cached context (prompts served in chunks, prefixes shared by a fork)
        {"name": "prefill chunks paged", "op": "prefill", "mode": "paged", "seqs": 4, "longest": 6000, **g8, "page": 16, "type": "bf16"},
        # parallel samples of a few prompts: shared pages, one partial page copied for each child
        {"name": "pages fork", "op": "pages", "mode": "fork", "seqs": 24, "longest": 900, "planes": 32, **g4, "page": 16, "type": "bf16"},
        # a pool after much freeing: live pages move to the front
        {"name": "pages compact", "op": "pages", "mode": "compact", "seqs": 40, "longest": 1024, "planes": 32, **g4, "page": 64, "type": "f16"},
    ]


def _spread(rng, low, high):
    """A whole number, its logarithm spread evenly."""
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill", "prefill", "pages"])
    hq, hkv, d = rng.choice(HEADS)
    case = {"op": op, "hq": hq, "hkv": hkv, "d": d, "page": rng.choice(PAGES), "type": rng.choice(["bf16", "f16"])}
    if op == "append":
        case["mode"] = rng.choice(["step", "prompt"])
        case["seqs"] = _spread(rng, 1, 256 if case["mode"] == "step" else 12)
        case["longest"] = _spread(rng, 2, 4096 if case["mode"] == "step" else 2048)
    elif op == "decode":
        case["seqs"] = _spread(rng, 1, 128)
        # all sequences together hold at most as many key channels as the largest listed case
        case["longest"] = _spread(rng, 1, min(131072, 16 * 32768 * 1024 // (case["seqs"] * hkv * d)))
    elif op == "prefill":
        case["mode"] = rng.choice(["packed", "paged"])
        case["seqs"] = _spread(rng, 1, 16)
        # scores of the padded batch: at most the largest listed case's
        case["longest"] = _spread(rng, 1, min(8192, int((8192 * 8192 * 32 / (case["seqs"] * hq)) ** 0.5)))
        case["page"] = case["page"] if case["mode"] == "paged" else 0
    else:
        case["mode"] = rng.choice(["fork", "compact"])
        case["seqs"] = _spread(rng, 3, 40)
        case["planes"] = 2 * _spread(rng, 1, 16)
        # the pool holds at most as much as the largest listed case's
        case["longest"] = _spread(rng, 20, max(24, min(1024, 40 * 1024 * 32 * 1024 // (case["seqs"] * case["planes"] * hkv * d))))
    return case


def _lengths(case):
    """Lengths of the case's sequences, the same for every seed: the longest is there, the others are ragged, and a
    batch of eight or more has empty slots and a sequence of one token."""
    n, longest = case["seqs"], case["longest"]
    rng = random.Random("%d %d %s" % (n, longest, case["op"]))
    got = [longest] + [rng.randint(max(1, longest // 4), longest) for _ in range(n - 1)]
    if n >= 8 and case["op"] in ("decode", "prefill"):
        got[-1], got[-2], got[-3] = 0, 1, 0
    rng.shuffle(got)
    return got


def _prefix(case):
    """Cached tokens before each sequence's new ones, for the paged prefill: a third to nearly all of its length."""
    rng = random.Random("prefix %d %d" % (case["seqs"], case["longest"]))
    return [int(n * rng.uniform(0.33, 0.95)) if n > 1 else 0 for n in _lengths(case)]


def _ceil(a, b):
    return -(-a // b)


def work(case):
    hq, hkv, d, lens = case["hq"], case["hkv"], case["d"], _lengths(case)
    if case["op"] == "append":
        tokens = case["seqs"] if case["mode"] == "step" else sum(lens)
        # the QKV rows in, rotated queries, keys and values out, one rotation row each, indexes
        return {"bytes": tokens * (4 * (hq + 2 * hkv) * d + 4 * d + 12), "flops": tokens * 3 * (hq + hkv) * d}
    if case["op"] == "decode":
        used = sum(lens)
        return {"bytes": 4 * used * hkv * d + 4 * case["seqs"] * hq * d + sum(4 * _ceil(n, case["page"]) for n in lens),
                "flops": 4 * used * hq * d}
    if case["op"] == "prefill":
        old = _prefix(case) if case["mode"] == "paged" else [0] * len(lens)
        new = sum(n - p for n, p in zip(lens, old))
        pairs = sum(n * (n + 1) // 2 - p * (p + 1) // 2 for n, p in zip(lens, old))
        return {"bytes": 4 * new * hq * d + 4 * sum(lens) * hkv * d, "flops": 4 * pairs * hq * d}
    row = 2 * case["planes"] * hkv * d  # one token in all planes
    if case["mode"] == "fork":
        pool = _pool(case)
        rest = sum(lens[p] % case["page"] for p in pool["parents"])
        return {"bytes": 2 * row * rest + 8 * pool["pages"] + 8 * len(lens) * _width(case), "flops": 0}
    pool = _pool(case)
    return {"bytes": 2 * row * case["page"] * len(_movers(pool)) + 12 * pool["pages"] + 8 * len(lens) * _width(case), "flops": 0}


# ----------------------------------------------------------------------------------------------------------
# inputs


def _width(case):
    return _ceil(max(_lengths(case)), case["page"]) + 1


def _pool(case):
    """Which pages of a pool are live, and who forks whom: from the case alone.  A third of the sequences (at least
    one) are parents; the last third are empty slots for children in "fork" and freed sequences in "compact"."""
    lens, page = _lengths(case), case["page"]
    n = len(lens)
    rng = random.Random("pool %d %d %s" % (n, case["longest"], case["mode"]))
    gone = set(range(n - max(1, n // 3), n)) if case["mode"] == "fork" else set(rng.sample(range(n), max(1, 2 * n // 5)))
    need = [_ceil(m, page) for m in lens]
    pages = sum(need) + max(4, sum(need) // 8) + n
    order = list(range(pages))
    rng.shuffle(order)
    rows, at = [], 0
    for s in range(n):
        rows.append(order[at:at + need[s]] if s not in gone else [])
        at += need[s]
    children = sorted(gone) if case["mode"] == "fork" else []
    parents = [i % max(1, n // 3) for i in range(len(children))]
    return {"pages": pages, "rows": rows, "gone": gone, "children": children, "parents": parents}


def _movers(pool):
    live = {p for r in pool["rows"] for p in r}
    return [p for p in live if p >= len(live)]


def _normal(g, shape, t, gain=1.0, shift=0.0):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    return x.mul_(gain).add_(shift).to(t)


def _keys_values(g, lead, hkv, tail, d, t):
    """Keys with a few strong channels, values with a mean of their own per channel, as trained models have them."""
    strong = 1.0 + 3.0 * (torch.rand((hkv, 1, d), generator=g, device=DEV) < 0.03)
    mean = 0.25 * torch.randn((hkv, 1, d), generator=g, device=DEV)
    k, v = (torch.empty((lead, hkv, tail, d), device=DEV, dtype=t) for _ in "kv")
    step = max(1, (1 << 27) // max(1, hkv * tail * d))
    for a in range(0, lead, step):
        n = min(step, lead - a)
        k[a:a + n] = torch.randn((n, hkv, tail, d), generator=g, device=DEV).mul_(strong).to(t)
        v[a:a + n] = torch.randn((n, hkv, tail, d), generator=g, device=DEV).add_(mean).to(t)
    return k, v


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return _ints(at)


def _tables(g, case, lens):
    """Tables over a shuffled pool with some pages to spare; unused entries are -1."""
    page, width = case["page"], _width(case)
    need = torch.tensor([_ceil(n, page) for n in lens], device=DEV)
    total = int(sum(_ceil(n, page) for n in lens))
    pages = total + max(3, total // 16)
    order = torch.randperm(pages, generator=g, device=DEV)
    col = torch.arange(width, device=DEV)[None]
    at = (torch.cumsum(need, 0) - need)[:, None] + col
    return torch.where(col < need[:, None], order[at.clamp(max=pages - 1)], -1).to(torch.int32), pages


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    t = TYPES[case["type"]]
    hq, hkv, d, lens = case["hq"], case["hkv"], case["d"], _lengths(case)
    s = dict(case, lens_host=lens, scale=d ** -0.5)
    if case["op"] == "append":
        if case["mode"] == "step":
            seq, pos = list(range(len(lens))), [n - 1 for n in lens]
        else:
            seq = [i for i, n in enumerate(lens) for _ in range(n)]
            pos = [j for n in lens for j in range(n)]
        s["seq"], s["pos"] = _ints(seq), _ints(pos)
        s["qkv"] = _normal(g, (len(seq), (hq + 2 * hkv) * d), t)
        s["tables"], pages = _tables(g, case, lens)
        s["k_pages"], s["v_pages"] = _keys_values(g, pages, hkv, case["page"], d, t)
        # one row for each position: the cosines, then the sines, of position * 10000^(-2i/D)
        rate = 10000.0 ** (-torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d)
        angle = torch.arange(case["longest"], device=DEV, dtype=torch.float64)[:, None] * rate
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    elif case["op"] == "decode":
        s["q"] = _normal(g, (len(lens), hq, d), t, 1.5)
        s["tables"], pages = _tables(g, case, lens)
        s["k_pages"], s["v_pages"] = _keys_values(g, pages, hkv, case["page"], d, t)
        s["lens"] = _ints(lens)
    elif case["op"] == "prefill":
        old = _prefix(case) if case["mode"] == "paged" else [0] * len(lens)
        new = [n - p for n, p in zip(lens, old)]
        s["new_host"], s["cu_q"], s["lens"] = new, _starts(new), _ints(lens)
        if case["mode"] == "paged":
            s["q"] = _normal(g, (sum(new), hq, d), t, 1.5)
            s["tables"], pages = _tables(g, case, lens)
            s["k_pages"], s["v_pages"] = _keys_values(g, pages, hkv, case["page"], d, t)
        else:
            # the three parts of one fused QKV output, as the linear leaves them
            qkv = _normal(g, (sum(lens), hq + 2 * hkv, d), t)
            qkv[:, :hq] *= 1.5
            qkv[:, hq + hkv:] += (0.25 * torch.randn((hkv, d), generator=g, device=DEV)).to(t)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        pool, width = _pool(case), _width(case)
        # which page holds what differs by seed: the ids of the live pages are shifted around the pool
        turn = int(torch.randint(0, pool["pages"], (1,), generator=g, device=DEV).item()) if case["mode"] == "fork" else 0
        rows = [[(p + turn) % pool["pages"] for p in r] for r in pool["rows"]]
        refs = [0] * pool["pages"]
        for r in rows:
            for p in r:
                refs[p] += 1
        s["tables"] = _ints([r + [-1] * (width - len(r)) for r in rows])
        s["refs"] = _ints(refs)
        s["lens"] = _ints([0 if i in pool["gone"] else n for i, n in enumerate(lens)])
        shape = (case["planes"], pool["pages"], hkv, case["page"], d)
        s["cache"] = torch.empty(shape, device=DEV, dtype=t)
        for plane in s["cache"]:
            plane.copy_(torch.randn(shape[1:], generator=g, device=DEV, dtype=torch.float32))
        s["refs_out"], s["tables_out"], s["lens_out"] = (torch.empty_like(s[k]) for k in ("refs", "tables", "lens"))
        if case["mode"] == "fork":
            s["parents"], s["children"] = _ints(pool["parents"]), _ints(pool["children"])
    return s


# ----------------------------------------------------------------------------------------------------------
# one pass


def run(s):
    if own:
        return _own(s)
    return {"append": _append, "decode": _decode, "prefill": _prefill, "pages": _pages}[s["op"]](s)


def _own(s):
    import quantized_linear_layers_awq_amd as tf

    if s["op"] == "append":
        q = tf.tf_kv_append(s["qkv"], s["rope"], s["seq"], s["pos"], s["tables"], s["k_pages"], s["v_pages"], s["hq"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["op"] == "decode":
        return tf.tf_attn_decode(s["q"], s["k_pages"], s["v_pages"], s["tables"], s["lens"], s["longest"], s["scale"])
    if s["op"] == "prefill" and s["mode"] == "packed":
        return tf.tf_attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_q"], s["longest"], s["scale"])
    if s["op"] == "prefill":
        return tf.tf_attn_prefill_paged(s["q"], s["k_pages"], s["v_pages"], s["tables"], s["cu_q"], s["lens"], max(s["new_host"]),
                                        s["scale"])
    if s["mode"] == "fork":
        short = tf.tf_kv_fork(s["cache"], s["refs"], s["tables"], s["lens"], s["parents"], s["children"],
                              refs_out=s["refs_out"], tables_out=s["tables_out"], lens_out=s["lens_out"])
        return {"cache": s["cache"].view(torch.int16), "refs": s["refs_out"], "tables": s["tables_out"], "lens": s["lens_out"],
                "status": short}
    moved = tf.tf_kv_compact(s["cache"], s["refs"], s["tables"], refs_out=s["refs_out"], tables_out=s["tables_out"])
    return {"cache": s["cache"].view(torch.int16), "refs": s["refs_out"], "tables": s["tables_out"], "moved": moved}


def _rotate(x, cos, sin):
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _append(s):
    hq, hkv, d, page = s["hq"], s["hkv"], s["d"], s["page"]
    x = s["qkv"].float().view(-1, hq + 2 * hkv, d)
    pos, seq = s["pos"].long(), s["seq"].long()
    cos, sin = s["rope"][pos][:, None].chunk(2, -1)
    q = _rotate(x[:, :hq], cos, sin).to(s["qkv"].dtype)
    at = s["tables"][seq, pos // page].long()
    s["k_pages"][at, :, pos % page] = _rotate(x[:, hq:hq + hkv], cos, sin).to(q.dtype)
    s["v_pages"][at, :, pos % page] = x[:, hq + hkv:].to(q.dtype)
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _gather(pages, tables, longest):
    """The first `longest` tokens of each sequence out of its pages, fp32 [seqs][Hkv][longest][D]."""
    x = pages[tables.clamp(min=0).long()]
    n, w, hkv, page, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, hkv, w * page, d)[:, :, :longest].float().contiguous()


def _softmax_product(q, k, v, keep):
    """softmax(q k^T) v over the kept keys, all of it fp32; a row that keeps none is zero.  q [n][h][G][D]."""
    x = torch.matmul(q, k.transpose(-1, -2).contiguous()).masked_fill_(~keep, LOWEST)
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    return torch.matmul(x, v) / torch.where(total > 0, total, 1.0)


def _decode(s):
    hkv, d = s["hkv"], s["d"]
    q = s["q"].float().view(len(s["q"]), hkv, -1, d) * s["scale"]
    longest = s["longest"]
    keep = torch.arange(longest, device=DEV)[None, None, None] < s["lens"][:, None, None, None]
    out = _softmax_product(q, _gather(s["k_pages"], s["tables"], longest), _gather(s["v_pages"], s["tables"], longest), keep)
    return out.reshape(s["q"].shape).to(s["q"].dtype)


def _padded(x, cu, longest):
    """Packed rows to a padded batch, and which of its rows are real."""
    at = cu[:-1, None].long() + torch.arange(longest, device=DEV)[None]
    real = at < cu[1:, None]
    return x[at.clamp(max=len(x) - 1)], real


def _prefill(s):
    hq, hkv, d, cu = s["hq"], s["hkv"], s["d"], s["cu_q"]
    q, real = _padded(s["q"], cu, max(s["new_host"]))
    n, lq = real.shape
    q = q.float().mul_(s["scale"]).view(n, lq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    if s["mode"] == "paged":
        k, v = (_gather(s[x], s["tables"], s["longest"]) for x in ("k_pages", "v_pages"))
    else:
        k, v = (_padded(s[x], cu, s["longest"])[0].float().permute(0, 2, 1, 3).contiguous() for x in ("k", "v"))
    # the last new token sees every key, the one before it one fewer, ...
    last = s["lens"][:, None] - (cu[1:] - cu[:-1])[:, None] + torch.arange(lq, device=DEV)[None]
    keep = torch.arange(s["longest"], device=DEV)[None, None] <= last[:, :, None]
    out = _softmax_product(q, k, v, keep[:, None].repeat(1, 1, hq // hkv, 1))
    out = out.view(n, hkv, hq // hkv, lq, d).permute(0, 3, 1, 2, 4).reshape(n, lq, hq, d)
    return out[real].to(s["q"].dtype)


def _pages(s):
    cache, refs, tables = s["cache"], s["refs"], s["tables"]
    pages, width = len(refs), tables.shape[1]
    col = torch.arange(width, device=DEV)[None]
    if s["mode"] == "fork":
        parents, children = s["parents"].long(), s["children"].long()
        size = s["lens"][parents]
        full, rest = (size // s["page"])[:, None], size % s["page"]
        free = torch.nonzero(refs == 0)[:, 0]
        need = torch.cumsum((rest > 0).int(), 0)
        fresh = free[(need - 1).clamp(min=0)]
        rows = tables[parents]
        row = torch.where(col < full, rows, torch.where((col == full) & (rest > 0)[:, None], fresh[:, None].int(), -1))
        tables_out, lens_out = tables.clone(), s["lens"].clone()
        tables_out[children], lens_out[children] = row, size
        used = row[row >= 0].long()
        refs_out = refs.clone().index_add_(0, used, torch.ones_like(used, dtype=torch.int32))
        part = torch.nonzero(rest > 0)[:, 0]
        source, to = rows.gather(1, full.long())[part, 0].long(), fresh[part]
        keep = torch.arange(s["page"], device=DEV)[None, None, None, :, None] < rest[part][None, :, None, None, None]
        cache[:, to] = torch.where(keep, cache[:, source], cache[:, to])
        short = (need[-1] - len(free)).clamp(min=0).int().view(1)
        return {"cache": cache.view(torch.int16), "refs": refs_out, "tables": tables_out, "lens": lens_out, "status": short}
    live = refs > 0
    at = torch.arange(pages, device=DEV)
    front = at < live.sum()
    source, to = torch.nonzero(live & ~front)[:, 0], torch.nonzero(~live & front)[:, 0]
    moved = torch.where(live, at, -1).int()
    moved[source] = to.int()
    cache[:, to] = cache[:, source]
    refs_out = torch.where(front & live, refs, 0)
    refs_out[to] = refs[source]
    tables_out = torch.where(tables >= 0, moved[tables.clamp(min=0).long()], -1)
    return {"cache": cache.view(torch.int16), "refs": refs_out, "tables": tables_out, "moved": moved}


# ----------------------------------------------------------------------------------------------------------
# the definitions, in fp64


def exact(case, seed):
    if case["op"] == "pages":  # pages are copied and numbered, not computed
        return None
    s = prepare(case, seed)
    hq, hkv, d, lens, page = s["hq"], s["hkv"], s["d"], s["lens_host"], s["page"]
    if s["op"] == "append":
        x = s["qkv"].double().view(-1, hq + 2 * hkv, d)
        # channel i < D/2 is the real part and channel i + D/2 the imaginary part of a number turned by the angle
        z = torch.complex(x[..., :d // 2], x[..., d // 2:])
        table = s["rope"].double()
        turn = torch.complex(table[:, :d // 2], table[:, d // 2:])[s["pos"].long()][:, None]
        y = torch.view_as_real(z * turn).movedim(-1, -2).reshape(x.shape)
        k, v = s["k_pages"].double(), s["v_pages"].double()
        flat = s["tables"][s["seq"].long(), torch.div(s["pos"], page, rounding_mode="floor").long()].long() * page + s["pos"] % page
        for h in range(hkv):
            for dst, src in ((k, y[:, hq + h]), (v, x[:, hq + hkv + h])):
                plane = dst[:, h].reshape(-1, d)
                plane[flat] = src
                dst[:, h] = plane.view(-1, page, d)
        return {"q": y[:, :hq], "k_pages": k, "v_pages": v}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    starts = s["cu_q"].tolist() if s["op"] == "prefill" else list(range(len(lens) + 1))
    for i, n in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        if n == 0 or a == b:
            continue
        for h in range(hkv):
            if "k_pages" in s:
                ids = s["tables"][i, :_ceil(n, page)].long()
                k, v = (s[x][ids, h].reshape(-1, d)[:n].double() for x in ("k_pages", "v_pages"))
            else:
                k, v = (s[x][a:b, h].double() for x in ("k", "v"))
            for j in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = s["q"][a:b, j].double() @ k.T * s["scale"]
                if s["op"] == "prefill":
                    x += torch.full_like(x, LOWEST).triu(n - (b - a) + 1)
                out[a:b, j] = torch.softmax(x, -1) @ v
    return out
