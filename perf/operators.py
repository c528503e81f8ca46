"""Grouped-query attention over a paged key-value cache, and that cache's upkeep:
the cases on which the operators are measured, each with a plain form.

  append   new tokens' keys and values written into their pages (bf16, fp32 or fp8 cache)
  decode   attention of single query tokens over the paged cache
  prompt   causal attention over whole prompts, packed one after the other
  pages    admitting sequences (free + extend), forking them, compacting the pool

Shapes: queries [rows, heads, dim]; caches [pages, kv heads, page size, dim];
page table [sequences, pages per sequence]; fp8 caches carry one fp32 scale
per cached row, [pages, kv heads, page size].
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}
SIZES = {"bf16": 2, "fp32": 4, "fp8": 1}
FP8_MAX = 448.0


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one decode step of a full batch: one new token a sequence, its key and value stored
        {"name": "append_decode_bf16", "op": "append", "n_seqs": 64, "most": 2048, "new": 1, "kv_heads": 8, "heads": 32,
         "dim": 128, "page": 64, "cache": "bf16"},
        # the keys and values of whole prompts (ragged, 16K tokens in all) rounded into an fp8 cache
        {"name": "append_prompt_fp8", "op": "append", "n_seqs": 11, "most": 2600, "new": 0, "kv_heads": 8, "heads": 32,
         "dim": 128, "page": 64, "cache": "fp8"},
        # a single user's next token at a short context: latency
        {"name": "decode_1row_bf16", "op": "decode", "n_seqs": 1, "tokens": 1, "most": 777, "ragged": False, "kv_heads": 8,
         "heads": 32, "dim": 128, "page": 64, "cache": "bf16"},
        # a batch of long contexts of different lengths: the cache's bytes
        {"name": "decode_32x32k_bf16", "op": "decode", "n_seqs": 32, "tokens": 1, "most": 32768, "ragged": True, "kv_heads": 8,
         "heads": 32, "dim": 128, "page": 64, "cache": "bf16"},
        # the same kind of batch over an fp8 cache, twice the sequences, twice the heads a group
        {"name": "decode_64x32k_fp8", "op": "decode", "n_seqs": 64, "tokens": 1, "most": 32768, "ragged": True, "kv_heads": 8,
         "heads": 64, "dim": 128, "page": 64, "cache": "fp8"},
        # a small model in fp32, several tokens a sequence verified at once, small pages, odd group
        {"name": "decode_fp32_odd", "op": "decode", "n_seqs": 5, "tokens": 3, "most": 5003, "ragged": True, "kv_heads": 3,
         "heads": 15, "dim": 64, "page": 16, "cache": "fp32"},
        # a handful of short prompts of a small model: latency and raggedness
        {"name": "prompt_short_bf16", "op": "prompt", "n_seqs": 7, "most": 300, "total": 901, "kv_heads": 4, "heads": 16,
         "dim": 64, "type": "bf16"},
        # a prefill batch of 16K tokens: one long prompt, the others shorter
        {"name": "prompt_16k_bf16", "op": "prompt", "n_seqs": 5, "most": 8192, "total": 16384, "kv_heads": 8, "heads": 32,
         "dim": 128, "type": "bf16"},
        # the parity type: a few prompts in fp32
        {"name": "prompt_fp32", "op": "prompt", "n_seqs": 3, "most": 1024, "total": 1800, "kv_heads": 4, "heads": 8, "dim": 64,
         "type": "fp32"},
        # a batch turns over: finished sequences give their pages back and new prompts take theirs
        {"name": "pages_admit", "op": "pages", "act": "admit", "n_seqs": 256, "take": 64, "most": 32768, "page": 64, "layers": 0,
         "kv_heads": 8, "dim": 128},
        # parallel sampling: 48 continuations branch off running sequences, each with its own last page in every layer
        {"name": "pages_fork", "op": "pages", "act": "fork", "n_seqs": 64, "take": 48, "most": 1500, "page": 64, "layers": 4,
         "kv_heads": 8, "dim": 128},
        # the pool is drawn together after most sequences left, so that its upper part can be given up
        {"name": "pages_compact", "op": "pages", "act": "compact", "n_seqs": 96, "take": 56, "most": 2000, "page": 64,
         "layers": 3, "kv_heads": 8, "dim": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prompt", "prompt", "pages"])
    if op == "append":
        return {"op": op, "n_seqs": _log(rng, 1, 128), "most": _log(rng, 16, 2600), "new": rng.choice([0, 1, 1, 3]),
                "kv_heads": rng.choice([1, 2, 3, 4, 8]), "heads": 24, "dim": rng.choice([64, 128]),
                "page": rng.choice([16, 32, 64, 128]), "cache": rng.choice(["bf16", "fp8", "fp32"])}
    if op == "decode":
        kv, cache = rng.choice([1, 2, 3, 4, 8]), rng.choice(["bf16", "bf16", "fp8", "fp32"])
        most = _log(rng, 1, 32768)
        n = min(_log(rng, 1, 64), max(1, 1500000 // (most * SIZES[cache])))       # no more bytes than the listed ones
        return {"op": op, "n_seqs": n, "tokens": rng.choice([1, 1, 1, 2, 4]) if n <= 16 else 1,
                "most": most, "ragged": rng.random() < 0.7, "kv_heads": kv,
                "heads": kv * rng.choice([1, 2, 4, 5, 7, 8, 16]), "dim": rng.choice([64, 128]),
                "page": rng.choice([16, 32, 64, 128]), "cache": cache}
    if op == "prompt":
        kind = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        n, kv = _log(rng, 1, 24), rng.choice([1, 2, 4, 8])
        most = _log(rng, 1, 8192 if kind == "bf16" else 1500)
        total = min(n * most, rng.randint(most, most + most // 2 + n))
        return {"op": op, "n_seqs": n, "most": most, "total": max(total, most), "kv_heads": kv, "heads": kv * rng.choice([1, 2, 3, 4]),
                "dim": rng.choice([64, 128]), "type": kind}
    n = rng.randint(8, 96)
    return {"op": op, "act": rng.choice(["admit", "fork", "compact"]), "n_seqs": n, "take": rng.randint(2, n // 2),
            "most": _log(rng, 20, 2000), "page": rng.choice([16, 32, 64, 128]), "layers": rng.randint(1, 3),
            "kv_heads": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128])}


def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lens(case):
    """Sequence lengths, of the case alone (the seed changes values and page places)."""
    r, n, most = _rng(case), case["n_seqs"], case["most"]
    if case["op"] == "prompt":
        # one prompt of the largest length; the rest of the tokens in unequal parts
        rest = case["total"] - most
        lens = [most]
        for i in range(n - 1):
            left = n - 1 - i
            part = rest if left == 1 else int(rest * min(1.0, r.uniform(0.3, 1.9) / left))
            part = max(0, min(part, most))
            lens.append(part)
            rest -= part
        r.shuffle(lens)
        return lens
    if not case.get("ragged", True):
        return [most] * n
    lens = [r.randint(max(1, most // 2), most) for _ in range(n)]
    lens[r.randrange(n)] = most
    return lens


def _up(a, b):
    return -(-a // b)


# ----------------------------------------------------------------- prepare --

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _table(lens, width, page, pool, g):
    """Page table [n, width]: random places in the pool for each sequence's pages, -1 behind them."""
    n = len(lens)
    counts = torch.tensor([_up(x, page) for x in lens], device="cuda")
    used = torch.arange(width, device="cuda") < counts[:, None]
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    rank = (torch.cumsum(used.reshape(-1), 0) - 1).clamp_(min=0).reshape(n, width)
    return torch.where(used, perm[rank], torch.full_like(perm[rank], -1)).contiguous()


def _quantise(x):
    """Rows of x [..., dim] as fp8 codes with one scale each: amax / 448."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / FP8_MAX, torch.ones_like(amax))
    return (x / scale[..., None]).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn), scale


def _pool(shape, kind, g):
    """A cache of random rows (and its scales where it is fp8)."""
    out = torch.empty(shape, dtype=DTYPES[kind], device="cuda")
    scale = torch.empty(shape[:-1], dtype=torch.float32, device="cuda") if kind == "fp8" else None
    step = max(1, (1 << 28) // max(1, math.prod(shape[1:])))
    for a in range(0, shape[0], step):
        x = torch.randn((min(step, shape[0] - a), *shape[1:]), generator=g, device="cuda")
        if kind == "fp8":
            out[a:a + step], scale[a:a + step] = _quantise(x)
        else:
            out[a:a + step] = x
    return out, scale


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "prompt":
        lens, h, kv, d = _lens(case), case["heads"], case["kv_heads"], case["dim"]
        total = sum(lens)
        # one fused projection's output; queries, keys and values are views of its rows
        qkv = torch.randn((total, h + 2 * kv, d), generator=g, device="cuda").to(DTYPES[case["type"]])
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        s.update(q=qkv[:, :h], k=qkv[:, h:h + kv], v=qkv[:, h + kv:], cu=cu,
                 cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), scale=1.0 / math.sqrt(d))
        return s
    lens, page = _lens(case), case["page"]
    if case["op"] == "pages":
        return _prepare_pages(case, s, lens, g)
    kv, d = case["kv_heads"], case["dim"]
    width = _up(case["most"], page)
    need = sum(_up(x, page) for x in lens)
    pool = need + 1 + need // 16
    s["table"] = _table(lens, width, page, pool, g)
    s["k_cache"], s["k_scale"] = _pool((pool, kv, page, d), case["cache"], g)
    s["v_cache"], s["v_scale"] = _pool((pool, kv, page, d), case["cache"], g)
    if case["op"] == "append":
        # `new` tokens at each sequence's end (0: the whole sequences), one of them a padded row
        batch, pos = [], []
        for b, x in enumerate(lens):
            first = 0 if case["new"] == 0 else max(0, x - case["new"])
            batch += [b] * (x - first)
            pos += range(first, x)
        if len(pos) > 1:
            pos[len(pos) // 2] = -1
        h = case["heads"]
        qkv = torch.randn((len(pos), h + 2 * kv, d), generator=g, device="cuda")
        qkv = qkv.to(torch.float32 if case["cache"] == "fp32" else torch.bfloat16)
        s.update(k=qkv[:, h:h + kv], v=qkv[:, h + kv:])
    else:
        # `tokens` rows a sequence, the last of them at its last token (positions before the first: empty rows)
        t = case["tokens"]
        batch = [b for b in range(len(lens)) for _ in range(t)]
        pos = [max(-1, x - t + i) for x in lens for i in range(t)]
        q = torch.randn((len(pos), case["heads"], d), generator=g, device="cuda")
        s["q"] = q.to(torch.float32 if case["cache"] == "fp32" else torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(d)
    s["row_batch"] = torch.tensor(batch, dtype=torch.int32, device="cuda")
    s["row_pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
    return s


def _prepare_pages(case, s, lens, g):
    """The pool's books. admit: `take` sequences are replaced by new ones; fork: the last `take` table rows are
    the branches of others; compact: the last `take` sequences have left and their pages lie free between the others'."""
    n, take, page = case["n_seqs"], case["take"], case["page"]
    width = _up(case["most"], page) + 1
    per = [_up(x, page) for x in lens]
    pool = sum(per) + take + 8
    table = _table(lens, width, page, pool, g)
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["act"] == "compact":
        table[n - take:] = -1
        length[n - take:] = 0
    count = torch.zeros(pool + 1, dtype=torch.int32, device="cuda")
    at = torch.where(table >= 0, table, pool).reshape(-1).long()
    count.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    s.update(table=table, length=length, count=count[:pool].contiguous())
    r = _rng(case)
    if case["act"] == "admit":
        s["seqs"] = torch.tensor(r.sample(range(n), take), dtype=torch.int32, device="cuda")
        s["add"] = torch.tensor([r.randint(1, case["most"] // 2 + 1) for _ in range(take)], dtype=torch.int32, device="cuda")
    if case["act"] == "fork":
        s["children"] = torch.arange(n - take, n, dtype=torch.int32, device="cuda")
        s["parents"] = torch.tensor([r.randrange(n - take) for _ in range(take)], dtype=torch.int32, device="cuda")
    if case["act"] != "admit":
        s["caches"] = [_pool((pool, case["kv_heads"], page, case["dim"]), "bf16", g)[0] for _ in range(2 * case["layers"])]
    return s


# --------------------------------------------------------------------- run --

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "append":
        return _append(s)
    if s["op"] == "decode":
        return _decode(s)
    if s["op"] == "prompt":
        return _prompt(s)
    if s["act"] == "admit":
        _free(s, s["seqs"].long())
        _extend(s, s["seqs"].long(), s["add"].long())
        return {"table": s["table"], "length": s["length"], "count": s["count"]}
    if s["act"] == "fork":
        _free(s, s["children"].long())
        _fork(s, s["parents"].long(), s["children"].long())
        return {"table": s["table"], "length": s["length"], "count": s["count"], "caches": s["caches"]}
    return _compact(s)


def _run_own(s):
    import sparse_attention_logits_b200 as dsa

    if s["op"] == "append":
        dsa.kv_cache_append(s["k"], s["v"], s["row_batch"], s["row_pos"], s["table"], s["k_cache"], s["v_cache"],
                            s["k_scale"], s["v_scale"])
        return _caches(s)
    if s["op"] == "decode":
        out, lse = dsa.gqa_decode_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["row_batch"], s["row_pos"],
                                            s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"out": out, "lse": lse}
    if s["op"] == "prompt":
        out, lse = dsa.gqa_prompt_attention(s["q"], s["k"], s["v"], s["cu_seqlens"], s["scale"])
        return {"out": out, "lse": lse}
    if s["act"] == "admit":
        dsa.kv_pages_free(s["table"], s["length"], s["count"], s["seqs"], s["page"])
        dsa.kv_pages_extend(s["table"], s["length"], s["count"], s["seqs"], s["add"], s["page"])
        return {"table": s["table"], "length": s["length"], "count": s["count"]}
    if s["act"] == "fork":
        dsa.kv_pages_free(s["table"], s["length"], s["count"], s["children"], s["page"])
        dsa.kv_pages_fork(s["table"], s["length"], s["count"], s["parents"], s["children"], s["page"], s["caches"])
        return {"table": s["table"], "length": s["length"], "count": s["count"], "caches": s["caches"]}
    table, count = dsa.kv_pages_compact(s["table"], s["count"], s["caches"])
    return {"table": table, "count": count, "caches": s["caches"]}


def _caches(s):
    out = {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["k_scale"] is not None:
        out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


def _append(s):
    pos, batch = s["row_pos"].long(), s["row_batch"].long()
    keep = pos >= 0
    pos, batch = pos[keep], batch[keep]
    page, slot = s["table"][batch, pos // s["page"]].long(), pos % s["page"]
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x[keep].float()
        if scale is not None:
            x, by = _quantise(x)
            scale[page, :, slot] = by
            cache.view(torch.uint8)[page, :, slot] = x.view(torch.uint8)
        else:
            cache[page, :, slot] = x.to(cache.dtype)
    return _caches(s)


def _gathered(cache, scale, pages):
    """[rows, kv heads, positions, dim] in 32 bits from the pages of each row."""
    x = cache.view(torch.uint8)[pages].view(cache.dtype) if scale is not None else cache[pages]
    x = x.float()
    if scale is not None:
        x *= scale[pages][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _decode(s):
    rows, h, d = s["q"].shape
    kv = s["kv_heads"]
    pages = s["table"][s["row_batch"].long()].clamp(min=0).long()
    q = s["q"].float().reshape(rows, kv, h // kv, d)
    z = (q @ _gathered(s["k_cache"], s["k_scale"], pages).transpose(2, 3)) * s["scale"]
    hidden = torch.arange(z.shape[-1], device=z.device) > s["row_pos"][:, None].long()
    z.masked_fill_(hidden[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    v = _gathered(s["v_cache"], s["v_scale"], pages).masked_fill_(hidden[:, None, :, None], 0.0)
    out = (p @ v) / total.clamp(min=1e-30)
    return {"out": out.reshape(rows, h, d).to(s["q"].dtype), "lse": (top + torch.log(total)).reshape(rows, h)}


def _prompt(s):
    q, k, v = (s[x].float() for x in "qkv")
    total, h, d = q.shape
    kv = k.shape[1]
    out = torch.empty_like(q)
    lse = torch.empty((total, h), dtype=torch.float32, device=q.device)
    for a, b in zip(s["cu"], s["cu"][1:]):          # each prompt by itself: a padded batch would work on padding
        n = b - a
        if n == 0:
            continue
        qs = q[a:b].reshape(n, kv, h // kv, d).permute(1, 2, 0, 3).reshape(kv, -1, d)
        z = (qs @ k[a:b].permute(1, 2, 0)).mul_(s["scale"]).reshape(kv, h // kv, n, n)
        at = torch.arange(n, device=q.device)
        z.masked_fill_(at > at[:, None], -math.inf)
        top = z.amax(-1, keepdim=True)
        p = z.sub_(top).exp_()
        sums = p.sum(-1, keepdim=True)
        o = (p.reshape(kv, -1, n) @ v[a:b].transpose(0, 1)).reshape(kv, h // kv, n, d) / sums
        out[a:b] = o.permute(2, 0, 1, 3).reshape(n, h, d)
        lse[a:b] = (top + torch.log(sums)).permute(2, 0, 1, 3).reshape(n, h)
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _held(s, seqs):
    """Which entries of these sequences' table rows are in use."""
    width = s["table"].shape[1]
    pages = (s["length"][seqs].long() + s["page"] - 1) // s["page"]
    return torch.arange(width, device=seqs.device) < pages[:, None]


def _add_refs(s, pages, used, by):
    n = s["count"].shape[0]
    count = torch.cat([s["count"], s["count"].new_zeros(1)])
    at = torch.where(used, pages.long(), n).reshape(-1)
    count.index_add_(0, at, torch.full_like(at, by, dtype=torch.int32))
    s["count"].copy_(count[:n])


def _free(s, seqs):
    _add_refs(s, s["table"][seqs], _held(s, seqs), -1)
    s["table"][seqs] = -1
    s["length"][seqs] = 0


def _free_pages(s):
    """The free pages' ids, lowest first (used pages' ids behind them)."""
    return torch.argsort((s["count"] > 0).to(torch.uint8), stable=True)


def _extend(s, seqs, add):
    have = (s["length"][seqs].long() + s["page"] - 1) // s["page"]
    want = (s["length"][seqs].long() + add + s["page"] - 1) // s["page"]
    need = want - have
    end = torch.cumsum(need, 0)
    fits = (end <= (s["count"] == 0).sum()) | (need == 0)
    rows = s["table"][seqs]
    j = torch.arange(rows.shape[1], device=seqs.device)
    fresh = (j >= have[:, None]) & (j < want[:, None]) & fits[:, None]
    order = _free_pages(s)
    rank = (end - need)[:, None] + j - have[:, None]
    rows = torch.where(fresh, order[rank.clamp(0, order.numel() - 1)].to(torch.int32), rows)
    s["table"][seqs] = rows
    s["length"][seqs] += torch.where(fits, add, torch.zeros_like(add)).to(torch.int32)
    _add_refs(s, rows, fresh, 1)


def _fork(s, parents, children):
    length = s["length"][parents]
    full, ends = length.long() // s["page"], length % s["page"] > 0
    order = _free_pages(s)
    rank = torch.cumsum(ends.long(), 0) - 1
    fresh = order[rank.clamp(min=0)].to(torch.int32)
    rows = s["table"][parents]
    j = torch.arange(rows.shape[1], device=parents.device)
    old = rows.gather(1, full[:, None].clamp(max=rows.shape[1] - 1))[:, 0]
    last = (j == full[:, None]) & ends[:, None]
    rows = torch.where(last, fresh[:, None], rows)
    s["table"][children] = rows
    s["length"][children] = length
    _add_refs(s, rows, (j < full[:, None]) | last, 1)
    src, dst = old[ends].long(), fresh[ends].long()
    for c in s["caches"]:
        c[dst] = c[src]


def _compact(s):
    n = s["count"].shape[0]
    used = s["count"] > 0
    ids = torch.arange(n, device=used.device)
    live = used.sum()
    src = torch.nonzero(used & (ids >= live))[:, 0]
    dst = torch.nonzero(~used & (ids < live))[:, 0]
    to = ids.clone()
    to[src] = dst
    for c in s["caches"]:
        c[dst] = c[src]
    table = torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()].to(torch.int32), s["table"])
    count = torch.where(ids < live, s["count"], torch.zeros_like(s["count"]))
    count[dst] = s["count"][src]
    return {"table": table, "count": count, "caches": s["caches"]}


# -------------------------------------------------------------------- work --

def work(case):
    lens = _lens(case)
    if case["op"] == "prompt":
        h, kv, d, e = case["heads"], case["kv_heads"], case["dim"], SIZES[case["type"]]
        total = sum(lens)
        return {"bytes": total * (2 * h + 2 * kv) * d * e + total * h * 4, "flops": sum(2 * h * d * n * (n + 1) for n in lens)}
    if case["op"] == "decode":
        h, kv, d, e = case["heads"], case["kv_heads"], case["dim"], SIZES[case["cache"]]
        row = 2 * kv * (d * e + (4 if case["cache"] == "fp8" else 0))
        t = case["tokens"]
        seen = sum(max(0, x - t + 1 + i) for x in lens for i in range(t))
        io = len(lens) * t * h * (2 * d * (4 if case["cache"] == "fp32" else 2) + 4)
        return {"bytes": sum(lens) * row + io, "flops": 4 * h * d * seen}
    if case["op"] == "append":
        kv, d, e = case["kv_heads"], case["dim"], SIZES[case["cache"]]
        n = sum(x if case["new"] == 0 else min(case["new"], x) for x in lens)
        e_in = 4 if case["cache"] == "fp32" else 2
        return {"bytes": n * 2 * kv * (d * (e + e_in) + (4 if case["cache"] == "fp8" else 0)) + 8 * n, "flops": 0}
    page, n, take = case["page"], case["n_seqs"], case["take"]
    width = _up(case["most"], page) + 1
    per = [_up(x, page) for x in lens]
    pool = sum(per) + take + 8
    data = 2 * case["layers"] * case["kv_heads"] * page * case["dim"] * 2
    r = _rng(case)
    if case["act"] == "admit":
        seqs = r.sample(range(n), take)
        new = [_up(r.randint(1, case["most"] // 2 + 1), page) for _ in range(take)]
        # table rows read and cleared, pages counted down; new entries written, pages counted up; the free pages found
        return {"bytes": sum(per[q] for q in seqs) * 16 + sum(new) * 12 + 4 * pool, "flops": 0}
    if case["act"] == "fork":
        parents = [r.randrange(n - take) for _ in range(take)]
        ends = sum(lens[p] % page > 0 for p in parents)
        return {"bytes": sum(per[p] for p in parents) * 32 + 2 * ends * data + 4 * pool, "flops": 0}
    live = sum(per[:n - take])
    moved = live * (pool - live) / pool              # the pages' places are random: this share lies above the live count
    return {"bytes": 2 * moved * data + 8 * pool + 8 * n * width, "flops": 0}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "pages":
        return _exact_pages(s)
    if case["op"] == "prompt":
        return _exact_prompt(s)
    return _exact_decode(s)


def _exact_append(s):
    """Codes are given as the unrounded quotient value / scale."""
    table = s["table"].tolist()
    rows = [(i, table[b][p // s["page"]], p % s["page"])
            for i, (b, p) in enumerate(zip(s["row_batch"].tolist(), s["row_pos"].tolist())) if p >= 0]
    i, pg, sl = (torch.tensor(x, device="cuda") for x in zip(*rows))
    out = {}
    for x, name in ((s["k"], "k"), (s["v"], "v")):
        cache = s[name + "_cache"].double()
        y = x[i].double()
        if s[name + "_scale"] is not None:
            scale = s[name + "_scale"].double()
            by = y.abs().max(-1).values / FP8_MAX
            by[by == 0] = 1.0
            scale[pg, :, sl] = by
            y = y / by[..., None]
            out[name + "_scale"] = scale
        cache[pg, :, sl] = y
        out[name + "_cache"] = cache
    return out


def _softmax_rows(z, v):
    """Attention of score rows z [..., positions] over v [..., positions, dim], with log sum exp."""
    lse = torch.logsumexp(z, -1)
    return torch.exp(z - lse[..., None]) @ v, lse


def _exact_decode(s):
    rows, h, d = s["q"].shape
    kv = s["kv_heads"]
    out = torch.zeros((rows, h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, h), -math.inf, dtype=torch.float64, device="cuda")
    for r, (b, p) in enumerate(zip(s["row_batch"].tolist(), s["row_pos"].tolist())):
        if p < 0:
            continue
        pages = s["table"][b, :p // s["page"] + 1].long()
        got = []
        for name in ("k", "v"):
            x = s[name + "_cache"].view(torch.uint8)[pages].view(s[name + "_cache"].dtype).double()
            if s[name + "_scale"] is not None:
                x = x * s[name + "_scale"][pages].double()[..., None]
            got.append(x.permute(1, 0, 2, 3).reshape(kv, -1, d)[:, :p + 1])
        z = torch.einsum("kgd,kpd->kgp", s["q"][r].double().reshape(kv, h // kv, d), got[0]) * s["scale"]
        o, m = _softmax_rows(z, got[1])
        out[r], lse[r] = o.reshape(h, d), m.reshape(h)
    return {"out": out, "lse": lse}


def _exact_prompt(s):
    total, h, d = s["q"].shape
    g = h // s["kv_heads"]
    out = torch.zeros((total, h, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((total, h), dtype=torch.float64, device="cuda")
    for a, b in zip(s["cu"], s["cu"][1:]):
        if a == b:
            continue
        future = torch.ones((b - a, b - a), dtype=torch.bool, device="cuda").triu(1)
        for i in range(h):
            z = s["q"][a:b, i].double() @ s["k"][a:b, i // g].double().T * s["scale"]
            out[a:b, i], lse[a:b, i] = _softmax_rows(z.masked_fill(future, -math.inf), s["v"][a:b, i // g].double())
    return {"out": out, "lse": lse}


def _exact_pages(s):
    """The books kept entry by entry; the pages' bytes moved accordingly."""
    table, count, page = s["table"].tolist(), s["count"].tolist(), s["page"]
    length = s["length"].tolist()
    src, dst = [], []

    def drop(q):
        for j in range(_up(length[q], page)):
            count[table[q][j]] -= 1
        table[q] = [-1] * len(table[q])
        length[q] = 0

    if s["act"] == "admit":
        seqs, add = s["seqs"].tolist(), s["add"].tolist()
        for q in seqs:
            drop(q)
        free = [i for i, c in enumerate(count) if c == 0]
        for q, a in zip(seqs, add):
            for j in range(_up(length[q], page), _up(length[q] + a, page)):
                table[q][j] = free.pop(0)
                count[table[q][j]] += 1
            length[q] += a
        return {"table": torch.tensor(table), "length": torch.tensor(length), "count": torch.tensor(count)}
    if s["act"] == "fork":
        for q in s["children"].tolist():
            drop(q)
        free = [i for i, c in enumerate(count) if c == 0]
        for p, q in zip(s["parents"].tolist(), s["children"].tolist()):
            table[q], length[q] = list(table[p]), length[p]
            if length[p] % page:
                j = length[p] // page
                src.append(table[p][j])
                dst.append(free.pop(0))
                table[q][j] = dst[-1]
            for j in range(_up(length[q], page)):
                count[table[q][j]] += 1
        out = {"length": torch.tensor(length)}
    else:
        live = sum(c > 0 for c in count)
        src = [i for i in range(live, len(count)) if count[i] > 0]
        dst = [i for i in range(live) if count[i] == 0]
        to = dict(zip(src, dst))
        table = [[to.get(x, x) for x in row] for row in table]
        for i, j in to.items():
            count[j], count[i] = count[i], 0
        out = {}
    caches = []
    for c in s["caches"]:
        x = c.double()
        x[dst] = c[src].double()
        caches.append(x)
    return dict(out, table=torch.tensor(table), count=torch.tensor(count), caches=caches)
