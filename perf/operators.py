"""Performance cases of the 8-bit paged K/V cache operators and of token sampling.

Three operators of a decode step, in the order a serving loop runs them:

* ``append``: rotate the new keys (and queries), round keys and values to
  8 bits with one scale per 16 tokens and head, and store them into a paged
  cache, rescaling the tokens a partly filled block already holds;
* ``attention``: ragged queries over that cache, o = softmax(q K^T s) V with
  keys [0, len) of every sequence, no mask among them (a block of a
  masked-diffusion decoder, or one token a sequence);
* ``sample``: one token a row from its logits with temperature, top-k, top-p
  and min-p, drawn with a given uniform number, and its probability.

``run`` with ``own`` false computes them with elementary torch operations, with
``own`` true through the library's entry points.
"""
from __future__ import annotations

import random

import numpy as np
import torch

own = False

PAGE = 64          # tokens per cache page
BLOCK = 16         # tokens that share a scale (one per head)
LIGHTEST = 2.0 ** -45   # a token lighter than this times the row's heaviest is never drawn
TINY_SCALE = 2.0 ** -100  # a scale below this is stored as 0 (all codes 0)

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}

# (query heads, K/V heads, head size, RoPE base) of the repository's models, and one generic
HEADS = {"llada": (32, 32, 128, 1e4), "dream": (28, 4, 128, 1e6), "small-gqa": (8, 2, 64, 1e6),
         "tiny": (4, 4, 32, 1e4), "gqa8": (64, 8, 128, 1e6)}
LLADA_VOCAB, DREAM_VOCAB, SMALL_VOCAB, TINY_VOCAB = 126464, 152064, 2051, 512


def _attn(name, heads, dtype, n, q, kv, ragged):
    return {"name": name, "op": "attention", "heads": heads, "dtype": dtype, "n_seqs": n,
            "q_len": q, "kv_len": kv, "ragged": ragged}


def _app(name, heads, dtype, n, new, old, ragged):
    return {"name": name, "op": "append", "heads": heads, "dtype": dtype, "n_seqs": n,
            "new_len": new, "old_len": old, "ragged": ragged}


def _samp(name, dtype, rows, vocab, k, p, minp, greedy):
    return {"name": name, "op": "sample", "dtype": dtype, "rows": rows, "vocab": vocab,
            "top_k": k, "top_p": p, "min_p": minp, "greedy": greedy}


def listed():
    return [
        # one token of one sequence after a 512-token context: what a lone user waits for
        _attn("attn-token-512", "dream", "bf16", 1, 1, 511, False),
        # a 32-token diffusion block near the end of the 1024 + 1024 generation
        _attn("attn-block-2k", "llada", "bf16", 1, 32, 2048, False),
        # batched serving: 16 sequences' blocks over contexts up to 1024 + 256
        _attn("attn-blocks-batch16", "llada", "f16", 16, 32, 1280, True),
        # 64 users, one token each, contexts up to 8K, one slot idle
        _attn("attn-tokens-batch64", "dream", "bf16", 64, 1, 8192, True),
        # a block over a context of 128K tokens, grouped heads (compute-bound)
        _attn("attn-block-128k", "dream", "bf16", 1, 32, 131055, False),
        # float32 model, odd ragged sizes, small heads
        _attn("attn-f32-odd", "small-gqa", "f32", 3, 7, 1333, True),
        # one new token for each of 64 users: blocks of 16 partly filled
        _app("append-tokens-batch64", "dream", "bf16", 64, 1, 1021, True),
        # a diffusion step's block for each of 16 sequences, at odd positions
        _app("append-blocks-batch16", "llada", "f16", 16, 32, 1003, True),
        # a long prompt enters the cache
        _app("append-prompt-8k", "llada", "bf16", 1, 8191, 0, False),
        # one row, all filters (a lone user's next token)
        _samp("sample-1-dream", "f32", 1, DREAM_VOCAB, 50, 0.95, 0.02, False),
        # a block's 32 masked positions with nucleus sampling
        _samp("sample-32-llada", "f32", 32, LLADA_VOCAB, 0, 0.9, 0.0, False),
        # 16 sequences' blocks at once, 16-bit logits, per-row filters, some rows greedy
        _samp("sample-512-llada", "bf16", 512, LLADA_VOCAB, 200, 0.95, 0.01, True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("attention", "append", "sample"))
    dtype = rng.choice(("bf16", "f16", "f32"))
    if op == "sample":
        return {"op": op, "dtype": dtype, "rows": _log(rng, 1, 384),
                "vocab": rng.choice((LLADA_VOCAB, DREAM_VOCAB, SMALL_VOCAB, TINY_VOCAB,
                                     _log(rng, 100, 152064))),
                "top_k": rng.choice((0, 1, _log(rng, 2, 4000))),
                "top_p": rng.choice((1.0, round(rng.uniform(0.05, 0.999), 3))),
                "min_p": rng.choice((0.0, round(rng.uniform(0.001, 0.3), 4))),
                "greedy": rng.random() < 0.3}
    heads = rng.choice(tuple(HEADS))
    hq, hkv, hd, _ = HEADS[heads]
    ragged = rng.random() < 0.7
    n = _log(rng, 1, 64)
    if op == "append":
        new = rng.choice((1, _log(rng, 2, 64), _log(rng, 64, 8191)))
        new = max(1, min(new, (8191 * 32 * 128) // (n * hkv * hd)))
        old = rng.choice((0, _log(rng, 1, 4096)))
        return {"op": op, "heads": heads, "dtype": dtype, "n_seqs": n, "new_len": new,
                "old_len": old, "ragged": ragged}
    q = rng.choice((1, _log(rng, 2, 80)))
    # within the largest listed cases: cached values read, and multiply-adds
    most = min(64 * 8192 * 4 * 128 // (n * hkv * hd), 32 * 131055 * 28 * 128 // (n * q * hq * hd))
    if dtype == "f32":
        most //= 4
    return {"op": op, "heads": heads, "dtype": dtype, "n_seqs": n, "q_len": q,
            "kv_len": _log(rng, 1, max(1, min(131072, most))), "ragged": ragged}


# ---------------------------------------------------------------- sizes of a case
def _lengths(case):
    """Rows and context of every sequence (Python lists): the case's alone, so that every
    seed has the same amount of work.  Ragged: anything from one token up, an idle slot
    without rows and one without context where there are four sequences or more."""
    n, ragged = case["n_seqs"], case["ragged"]
    rows = case["q_len"] if case["op"] == "attention" else case["new_len"]
    ctx = case["kv_len"] if case["op"] == "attention" else case["old_len"]
    r = random.Random(1000003 * n + 1009 * rows + ctx)
    a, b = [rows] * n, [ctx] * n
    if ragged:
        a = [rows] + [r.randint(max(1, rows // 2), rows) for _ in range(n - 1)]
        b = [ctx] + [r.randint(min(1, ctx), ctx) for _ in range(n - 1)]
        if n >= 4:
            a[n // 2] = 0
            b[n // 3] = 0
    return a, b


def _pages(tokens):
    return -(-tokens // PAGE)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)


def _cache(g, case, lens, hkv, hd):
    """A paged cache whose pages lie in random order, filled with codes of Gaussian keys and
    values whose size changes from block to block."""
    n = len(lens)
    width = max(1, max(_pages(x) for x in lens))
    pages = sum(_pages(x) for x in lens) + 3
    dev = "cuda"
    table = torch.full((n, width), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu()
    at = 0
    for i, x in enumerate(lens):
        m = _pages(x)
        table[i, :m] = order[at:at + m]
        at += m
    st = {"table": table.to(dev)}
    for name in ("k", "v"):
        codes = torch.empty(pages, hkv, PAGE, hd, dtype=torch.int8, device=dev)
        scale = torch.empty(pages, hkv, PAGE // BLOCK, device=dev)
        part = max(1, (1 << 27) // (hkv * PAGE * hd))
        for p in range(0, pages, part):
            x = torch.randn(min(part, pages - p), hkv, PAGE // BLOCK, BLOCK * hd, generator=g, device=dev)
            top = x.abs().amax(-1)
            codes[p:p + part] = torch.round(x * (127.0 / top)[..., None]).to(torch.int8).view(-1, hkv, PAGE, hd)
            grow = torch.exp(0.3 * torch.randn(top.shape, generator=g, device=dev))
            scale[p:p + part] = top / 127.0 * grow
        st[name], st[name + "_scale"] = codes, scale
    return st


def _starts(rows):
    return torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")


def _rope(length, hd, theta):
    """(cos, sin) of every position and pair, angles in 64 bits."""
    inv = torch.pow(torch.tensor(theta, dtype=torch.float64),
                    -2.0 * torch.arange(hd // 2, dtype=torch.float64) / hd).cuda()
    a = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def prepare(case, seed):
    g, dt = _gen(seed), TYPES[case["dtype"]]
    dev = "cuda"
    if case["op"] == "sample":
        R, V = case["rows"], case["vocab"]
        x = torch.randn(R, V, generator=g, device=dev) * 2.5
        # a few candidates stand out, as under a trained head
        top = torch.randint(0, V, (R, 40), generator=g, device=dev)
        x.scatter_add_(1, top, 9.0 * torch.rand(R, 40, generator=g, device=dev))
        some = torch.rand(R, generator=g, device=dev)

        def per_row(value, off):   # every row its own setting; in some rows the filter is off
            near = value * (0.5 + torch.rand(R, generator=g, device=dev))
            return torch.where(torch.rand(R, generator=g, device=dev) < 0.1, torch.full_like(near, off), near)

        temp = 0.3 + 1.2 * torch.rand(R, generator=g, device=dev)
        if case["greedy"]:
            temp = torch.where(some < 0.25, torch.zeros_like(temp), temp)
        st = {"logits": x.to(dt), "temperature": temp, "mask_id": V - 1,
              "u": torch.rand(R, generator=g, device=dev, dtype=torch.float64),
              "top_k": None, "top_p": None, "min_p": None}
        if case["top_k"] > 0:
            st["top_k"] = per_row(case["top_k"], 0.0).round().to(torch.int32)
        if case["top_p"] < 1:
            st["top_p"] = per_row(case["top_p"], 1.0).clamp(max=1.0)
        if case["min_p"] > 0:
            st["min_p"] = per_row(case["min_p"], 0.0)
        return {"op": "sample", **st}
    hq, hkv, hd, theta = HEADS[case["heads"]]
    rows, ctx = _lengths(case)
    T = sum(rows)
    if case["op"] == "attention":
        st = _cache(g, case, ctx, hkv, hd)
        st["q"] = (1.5 * torch.randn(T, hq, hd, generator=g, device=dev)).to(dt)
        st["starts"] = _starts(rows)
        st["lens"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
        st["max_q"], st["max_len"] = max(rows), max(ctx)
        return {"op": "attention", "hkv": hkv, **st}
    st = _cache(g, case, [a + b for a, b in zip(rows, ctx)], hkv, hd)
    # one projection's output holds q, k and v of a token side by side
    qkv = torch.randn(T, hq + 2 * hkv, hd, generator=g, device=dev) * torch.exp(
        0.5 * torch.randn(T, 1, 1, generator=g, device=dev))
    qkv = qkv.to(dt)
    st["q"], st["k_new"], st["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    st["starts"] = _starts(rows)
    st["lens"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    st["rope"] = _rope(max(a + b for a, b in zip(rows, ctx)) + 5, hd, theta)
    st["max_new"] = max(rows)
    return {"op": "append", "hkv": hkv, **st}


# ---------------------------------------------------------------- plain forms
def _plain_attention(st):
    q, table, lens, starts = st["q"], st["table"], st["lens"].long(), st["starts"].long()
    T, hq, hd = q.shape
    n, width = table.shape
    hkv = st["hkv"]
    rep, L = hq // hkv, width * PAGE
    at = table.clamp(min=0).long().reshape(-1)

    def dense(codes, scale):   # [n, hkv, L, hd] in 32 bits
        x = codes[at].view(-1, hkv, PAGE // BLOCK, BLOCK, hd).float() * scale[at][..., None, None]
        return x.view(n, width, hkv, PAGE, hd).permute(0, 2, 1, 3, 4).reshape(n, hkv, L, hd)

    most = st["max_q"]
    t = torch.arange(most, device=q.device)
    here = t < (starts[1:] - starts[:-1])[:, None]                      # [n, most]
    src = (starts[:-1, None] + t).clamp(max=max(T - 1, 0))
    qs = q[src].float().view(n, most, hkv, rep, hd).permute(0, 2, 3, 1, 4).reshape(n, hkv, rep * most, hd)
    s = torch.matmul(qs, dense(st["k"], st["k_scale"]).transpose(2, 3)) * hd ** -0.5
    live = (torch.arange(L, device=q.device) < lens[:, None])[:, None, None]
    s = s.masked_fill(~live, float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, dense(st["v"], st["v_scale"])) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.view(n, hkv, rep, most, hd).permute(0, 3, 1, 2, 4).reshape(n, most, hq, hd)
    return o[here].to(q.dtype)


def _rotate(x, rope, pos):
    h = x.shape[-1] // 2
    c, s = rope[pos, :, 0][:, None], rope[pos, :, 1][:, None]
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _plain_append(st):
    starts, lens, table = st["starts"].long(), st["lens"].long(), st["table"].long()
    T = st["k_new"].shape[0]
    t = torch.arange(T, device=table.device)
    seq = torch.bucketize(t, starts[1:], right=True)
    pos = lens[seq] + t - starts[seq]
    count = starts[1:] - starts[:-1]
    block = table[seq, pos // PAGE] * (PAGE // BLOCK) + pos % PAGE // BLOCK
    slot = pos % BLOCK
    q = _rotate(st["q"].float(), st["rope"], pos).to(st["q"].dtype)
    news = {"k": _rotate(st["k_new"].float(), st["rope"], pos), "v": st["v_new"].float()}
    out = {"q": q}
    n_blocks = st["k"].shape[0] * (PAGE // BLOCK)
    first = torch.full((n_blocks,), -1, dtype=torch.long, device=t.device)
    owner = torch.zeros(n_blocks, dtype=torch.long, device=t.device)
    first[block] = pos - slot
    owner[block] = seq
    touched = (first >= 0).nonzero()[:, 0]
    place = first[touched][:, None] + torch.arange(BLOCK, device=t.device)
    own_len, own_new = lens[owner[touched]], count[owner[touched]]
    # old tokens of a touched block: before the new ones (all of this call's are appended)
    kept = (place < own_len[:, None]) & ~((place >= own_len[:, None]) & (place < (own_len + own_new)[:, None]))
    any_kept = kept.any(1)[:, None]
    for name, x in news.items():
        hkv, hd = x.shape[1:]
        size = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
        top = torch.zeros(n_blocks, hkv, device=x.device).scatter_reduce(0, block[:, None].expand_as(size), size, "amax")
        page, sub = touched // (PAGE // BLOCK), touched % (PAGE // BLOCK)
        old = torch.where(any_kept, st[name + "_scale"][page, :, sub], torch.zeros((), device=x.device))
        new = torch.maximum(old, top[touched] * (1.0 / 127.0))
        new = torch.where(new < TINY_SCALE, torch.zeros_like(new), new)
        st[name + "_scale"][page, :, sub] = new
        ratio = torch.where(new > 0, old / new, torch.zeros_like(new))[:, :, None, None]
        pool = st[name].view(-1, hkv, PAGE // BLOCK, BLOCK, hd)
        was = pool[page, :, sub].float()                                  # [blocks, hkv, 16, hd]
        pool[page, :, sub] = torch.where(kept[:, None, :, None], torch.round(was * ratio), was).to(torch.int8)
        full = torch.zeros(n_blocks, hkv, device=x.device)
        full[touched] = new
        mine = full[block][..., None]
        code = x * torch.where(mine > 0, torch.ones_like(mine) / mine, torch.zeros_like(mine))
        code = torch.where(torch.isnan(code), torch.zeros_like(code), torch.round(code)).clamp(-127, 127)
        pool[block // (PAGE // BLOCK), :, block % (PAGE // BLOCK), slot] = code.to(torch.int8)
        out[name] = (code * mine).to(st["q"].dtype)
        out[name + "_codes"], out[name + "_scale"] = st[name], st[name + "_scale"]
    return out


def _plain_sample(st):
    x = st["logits"].double()
    R, V = x.shape
    low = float("-inf")
    x = torch.where(torch.isnan(x), torch.full_like(x, low), x)
    x[:, st["mask_id"]] = low
    z, order = torch.sort(x, dim=1, descending=True, stable=True)
    temp = st["temperature"].double()[:, None]
    greedy = ~(temp > 0)
    top = z[:, :1]
    d = (z - top) / torch.where(greedy, torch.ones_like(temp), temp)
    e = torch.where(z == top, torch.ones_like(d), torch.exp(d))
    e = torch.where((z > low) & (e >= LIGHTEST), e, torch.zeros_like(e))
    rank = torch.arange(V, device=x.device)
    keep = z > low
    if st["top_k"] is not None:
        k = st["top_k"][:, None]
        keep &= (k <= 0) | (rank < k)
    if st["top_p"] is not None:
        p = st["top_p"].double()[:, None]
        w = e * keep
        before = torch.cumsum(w, 1) - w
        keep &= (p >= 1) | (before < p * w.sum(1, keepdim=True)) | (rank == 0)
    if st["min_p"] is not None:
        mp = st["min_p"].double()[:, None]
        keep &= (mp <= 0) | (e >= mp.clamp(max=1))
    w = torch.zeros_like(e).scatter(1, order, e * keep)
    c = torch.cumsum(w, 1)
    total = c[:, -1:]
    tok = (c <= st["u"].clamp(min=0)[:, None] * total).sum(1, keepdim=True)
    last = torch.where(w > 0, rank, torch.zeros_like(rank)).amax(1, keepdim=True)
    tok = torch.where(greedy, order[:, :1], torch.minimum(tok, last))
    prob = w.gather(1, tok) / total
    empty = top == low
    tok = torch.where(empty, torch.full_like(tok, -1), tok)
    prob = torch.where(empty, torch.zeros_like(prob), prob)
    return {"tok": tok[:, 0].to(torch.int32), "prob": prob[:, 0].float()}


# ---------------------------------------------------------------- one pass
def _handle(st):
    """The cache object a program makes once and keeps."""
    from kv_cache_decode_dualcache_b200 import fdllm
    if "cache" not in st:
        st["cache"] = fdllm.Kv8Cache(st["k"], st["v"], st["k_scale"], st["v_scale"], st["table"])
    return fdllm, st["cache"]


def run(state):
    op = state["op"]
    if not own:
        plain = {"attention": _plain_attention, "append": _plain_append, "sample": _plain_sample}
        return plain[op](state)
    if op == "attention":
        fdllm, cache = _handle(state)
        return fdllm.fdllm_kv8_attention(cache, state["q"], state["starts"], state["lens"],
                                         max_q=state["max_q"], max_len=state["max_len"])
    if op == "append":
        fdllm, cache = _handle(state)
        q, k, v = fdllm.fdllm_kv8_append(cache, state["k_new"], state["v_new"], state["starts"],
                                         state["lens"], rope=state["rope"], q=state["q"],
                                         max_new=state["max_new"], stored=True)
        return {"q": q, "k": k, "v": v, "k_codes": state["k"], "v_codes": state["v"],
                "k_scale": state["k_scale"], "v_scale": state["v_scale"]}
    from kv_cache_decode_dualcache_b200 import fdllm
    tok, prob = fdllm.fdllm_sample(state["logits"], state["u"], temperature=state["temperature"],
                                   top_k=state["top_k"], top_p=state["top_p"],
                                   min_p=state["min_p"], mask_id=state["mask_id"])
    return {"tok": tok, "prob": prob}


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "sample":
        R, V = case["rows"], case["vocab"]
        return {"bytes": R * V * e + R * 32, "flops": 4.0 * R * V}
    hq, hkv, hd, _ = HEADS[case["heads"]]
    rows, ctx = _lengths(case)
    T = sum(rows)
    if case["op"] == "attention":
        read = sum(c for r, c in zip(rows, ctx) if r)
        cached = read * hkv * 2 * hd + _pages(read) * (PAGE // BLOCK) * hkv * 8
        pairs = sum(r * c for r, c in zip(rows, ctx))
        return {"bytes": cached + 2 * T * hq * hd * e, "flops": 4.0 * pairs * hq * hd}
    moved = T * ((2 * hq + 4 * hkv) * hd * e + 2 * hkv * hd)   # rows in, rows out, codes
    scales = (T / BLOCK + case["n_seqs"]) * hkv * 8
    kept = sum(c % BLOCK for r, c in zip(rows, ctx) if r) * hkv * hd * 2
    table = len({c + i for r, c in zip(rows, ctx) for i in range(r)}) * hd * 4
    return {"bytes": moved + scales + kept + table, "flops": T * hd * (8.0 * hkv + 3.0 * hq)}


# ---------------------------------------------------------------- in 64 bits
def _exact_attention(st):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    hq, hd = st["q"].shape[1:]
    hkv = st["hkv"]
    starts, lens, table = st["starts"].tolist(), st["lens"].tolist(), st["table"].long()
    for i, L in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        if a == b or L == 0:
            continue
        pages = table[i, :_pages(L)]
        for h in range(hkv):
            k, v = (torch.einsum("pbtd,pb->pbtd", st[x][pages, h].double().view(-1, PAGE // BLOCK, BLOCK, hd),
                                 st[x + "_scale"][pages, h].double()).reshape(-1, hd)[:L] for x in ("k", "v"))
            group = slice(h * hq // hkv, (h + 1) * hq // hkv)
            x = torch.einsum("thd,ld->thl", st["q"][a:b, group].double(), k) / hd ** 0.5
            out[a:b, group] = torch.einsum("thl,ld->thd", torch.softmax(x, -1), v)
    return out


def _exact_append(st, dtype):
    rope = st["rope"].double()
    starts, lens = st["starts"].tolist(), st["lens"].tolist()
    dev = "cuda"
    k_new, v_new, q = (st[x].double() for x in ("k_new", "v_new", "q"))
    half = q.shape[-1] // 2
    turn = torch.complex(rope[..., 0], rope[..., 1])
    res = {x: torch.empty_like(y) for x, y in (("q", q), ("k", k_new), ("v", v_new))}
    scales = {x: st[x + "_scale"].double() for x in ("k", "v")}
    for i, L in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        if a == b:
            continue
        w = turn[L:L + b - a][:, None]

        def turned(x):
            z = torch.complex(x[..., :half], x[..., half:]) * w
            return torch.cat([z.real, z.imag], -1)

        res["q"][a:b] = turned(q[a:b])
        lead = L % BLOCK                      # old tokens of the first block
        for name, x in (("k", turned(k_new[a:b])), ("v", v_new[a:b])):
            blocks = -(-(lead + b - a) // BLOCK)
            y = torch.zeros(blocks * BLOCK, *x.shape[1:], dtype=torch.float64, device=dev)
            y[lead:lead + b - a] = x
            y = y.view(blocks, BLOCK, *x.shape[1:])
            top = y.abs().amax((1, 3)) / 127.0                                   # [blocks, hkv]
            at = torch.arange(blocks, device=dev) + L // BLOCK
            page, sub = st["table"][i].long()[at // (PAGE // BLOCK)], at % (PAGE // BLOCK)
            if lead:
                top[0] = torch.maximum(top[0], scales[name][page[0], :, sub[0]])
            scales[name][page, :, sub] = top
            s = top[:, None, :, None]
            y = torch.round(y / s).clamp(-127, 127) * s
            res[name][a:b] = y.reshape(-1, *x.shape[1:])[lead:lead + b - a]
    # The codes and, in 32 bits, what they stand for hang on which side of a half step a
    # product falls: defined by the operator's 32-bit products, they have no value in 64 bits.
    return {"q": res["q"], "k": res["k"] if dtype != "f32" else None,
            "v": res["v"] if dtype != "f32" else None, "k_codes": None, "v_codes": None,
            "k_scale": scales["k"], "v_scale": scales["v"]}


def _exact_sample(st):
    R, V = st["logits"].shape
    x = st["logits"].double().cpu().numpy()
    per = {n: (st[n].double().cpu().numpy() if st[n] is not None else None)
           for n in ("temperature", "top_k", "top_p", "min_p", "u")}
    tok, prob = np.full(R, -1, np.int32), np.zeros(R)
    for r in range(R):
        z = x[r].copy()
        z[st["mask_id"]] = -np.inf
        z[np.isnan(z)] = -np.inf
        best = int(np.argmax(z))
        if z[best] == -np.inf:
            continue
        T = per["temperature"][r]
        with np.errstate(invalid="ignore"):
            w = np.exp((z - z[best]) / (T if T > 0 else 1.0))
        w[w < LIGHTEST] = 0.0
        live = np.nonzero(w)[0]
        # heaviest first, the lower id first among equal logits
        live = live[np.lexsort((live, -z[live]))]
        if per["top_k"] is not None and per["top_k"][r] > 0:
            live = live[:int(per["top_k"][r])]
        if per["top_p"] is not None and per["top_p"][r] < 1:
            run_sum = np.cumsum(w[live])
            live = live[:max(1, int(np.searchsorted(run_sum, per["top_p"][r] * run_sum[-1], "left")) + 1)]
        if per["min_p"] is not None and per["min_p"][r] > 0:
            live = live[w[live] >= min(per["min_p"][r], 1.0)]
        ids = np.sort(live)
        total = np.cumsum(w[ids])
        pick = int(np.searchsorted(total, per["u"][r] * total[-1], "right"))
        tok[r] = best if not T > 0 else ids[min(pick, len(ids) - 1)]
        prob[r] = w[tok[r]] / total[-1]
    return {"tok": torch.from_numpy(tok), "prob": torch.from_numpy(prob)}


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "attention":
        return _exact_attention(st)
    if st["op"] == "append":
        return _exact_append(st, case["dtype"])
    return _exact_sample(st)
