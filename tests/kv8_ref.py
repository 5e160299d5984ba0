"""Plain implementations of the 8-bit cache operators and of sampling for the
tests: float64 on the CPU (the append's codes in the float32 steps that define
them), one sequence, block or row at a time."""
from __future__ import annotations

import numpy as np
import torch

PAGE, BLOCK = 64, 16


def make_cache(gen, lens, hkv, hd, spare=3, extra_width=1, device="cpu"):
    """Cache tensors for sequences of `lens` tokens whose pages lie in random
    order.  What no token occupies is hostile: scales NaN, table entries out
    of range."""
    n = len(lens)
    need = [-(-x // PAGE) for x in lens]
    n_pages = sum(need) + spare
    table = torch.full((n, max(need + [0]) + extra_width), 1 << 30, dtype=torch.int32)
    table[1::2] = torch.where(table[1::2] > 0, -7, 0).to(torch.int32)
    order = torch.randperm(n_pages, generator=gen)
    k = torch.randint(-127, 128, (n_pages, hkv, PAGE, hd), generator=gen).to(torch.int8)
    v = torch.randint(-127, 128, (n_pages, hkv, PAGE, hd), generator=gen).to(torch.int8)
    ks = torch.full((n_pages, hkv, PAGE // BLOCK), float("nan"))
    vs = ks.clone()
    at = 0
    for i, x in enumerate(lens):
        for j in range(need[i]):
            page = int(order[at])
            at += 1
            table[i, j] = page
            live = min(PAGE // BLOCK, -(-(x - j * PAGE) // BLOCK))
            for s in (ks, vs):
                s[page, :, :live] = torch.exp(torch.randn(hkv, live, generator=gen)) / 60
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs, "table": table}


def dense(cache, which, seq, L):
    """float64 [hkv, L, hd] of one sequence."""
    pages = cache["table"][seq, :-(-L // PAGE)].long()
    code = cache[which][pages].double()
    s = cache[which + "_scale"][pages].double().repeat_interleave(BLOCK, 2)[..., None]
    return (code * s).transpose(0, 1).flatten(1, 2)[:, :L]


def attention(cache, q, starts, lens, scale):
    """float64 (out, size, reach, grain): the attention, and the sizes its
    rounding errors scale with: sum_j p_j |v_j|, the row's largest
    sum_d |q_d k_d| scale, and max_j(p_j vs_j) sum_j |code_j|."""
    T, H, hd = q.shape
    out = torch.full((T, H, hd), float("nan"), dtype=torch.float64)
    size, reach, grain = torch.zeros_like(out), torch.zeros(T, H, 1, dtype=torch.float64), torch.zeros_like(out)
    hkv = cache["k"].shape[1]
    for i, L in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        if a == b:
            continue
        if L == 0:
            out[a:b] = 0.0
            continue
        k, v = dense(cache, "k", i, L), dense(cache, "v", i, L)
        ones = {"v": torch.ones_like(cache["v"]), "v_scale": cache["v_scale"], "table": cache["table"]}
        codes = {"v": cache["v"], "v_scale": torch.ones_like(cache["v_scale"]), "table": cache["table"]}
        vs, vc = dense(ones, "v", i, L)[..., 0], dense(codes, "v", i, L)
        for h in range(H):
            g = h // (H // hkv)
            x = q[a:b, h].double()
            p = torch.softmax(x @ k[g].T * scale, -1)
            out[a:b, h] = p @ v[g]
            size[a:b, h] = p @ v[g].abs()
            grain[a:b, h] = (p * vs[g]).amax(-1, keepdim=True) * vc[g].abs().sum(0)
            reach[a:b, h] = (x.abs() @ k[g].abs().T * abs(scale)).amax(-1, keepdim=True)
    return out, size, reach, grain


def attention_tol(size, reach, grain, want, L, hd, dtype):
    """Largest error of an output element that the kernel's roundings allow.

    Weights: exp2 is good to 2^-22; one fp16 term rounds a weight by 2^-11
    relative (half a step), two terms by 2^-21; and as fp16 steps are at least
    2^-24, each weight is off by up to 2^-25 however small it is.  Weights are
    w_j = c p_j vs_j with the largest at least 2^8 (2^W_EXP at the reference),
    so 1 / c <= 2^-8 max_j(p_j vs_j), and sum_j 2^-25 |code_j| / c is at most
    2^-33 of grain (a weight taken against an earlier, smaller reference is
    scaled down later, its error with it).  Scores: a chain of hd / 16
    tensor-core steps truncates by up to 2^-23 of sum |q k| each, and its
    result, the factor and log2 of the scale round a few times more; fp32 q as
    two terms is off by 2^-21.  A score error d changes a weight by d and,
    through the sum, the result by at most 2 d.  Output sums: one truncation
    of 2^-23 a step of 16 keys.  The last rounding is half a step, which
    below the smallest normal number of the type is eps / 2 times that number
    (2^-25 in fp16)."""
    fi = torch.finfo(dtype)
    two = dtype == torch.float32
    weight = 2.0 ** (-21 if two else -11) + 2.0 ** -21
    score = reach * (hd / 16 + 8) * 2.0 ** -23 + (reach * 2.0 ** -21 if two else 0)
    sums = (L / 16 + 40) * 2.0 ** -23
    return size * (weight + 2 * score + sums) + grain * 2.0 ** -33 + want.abs().clamp(min=fi.smallest_normal) * fi.eps / 2


def rotate(x, rope, pos):
    """float32, every operation rounded on its own."""
    h = x.shape[-1] // 2
    c, s = rope[pos, :, 0][:, None], rope[pos, :, 1][:, None]
    a, b = x[..., :h].float(), x[..., h:].float()
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def append(cache, k, v, starts, lens, pos=None, rope=None, q=None):
    """Updates `cache` in place; returns {"q", "k", "v", "lens"} (k, v: what
    the cache now stands for; rows of no sequence stay NaN)."""
    T, hkv, hd = k.shape
    out = {"k": torch.full(k.shape, float("nan")).to(k.dtype), "lens": list(lens)}
    out["v"] = out["k"].clone()
    out["q"] = torch.full(q.shape, float("nan")).to(q.dtype) if q is not None else None
    for i in range(len(lens)):
        a, b = starts[i], starts[i + 1]
        w0 = lens[i] if pos is None else pos[i]
        w1 = w0 + b - a
        if a == b:
            continue
        out["lens"][i] = max(lens[i], w1)
        at = torch.arange(w0, w1)
        kr = rotate(k[a:b], rope, at) if rope is not None else k[a:b].float()
        if q is not None:
            out["q"][a:b] = (rotate(q[a:b], rope, at) if rope is not None else q[a:b].float()).to(q.dtype)
        for which, x in (("k", kr), ("v", v[a:b].float())):
            for blk in range(w0 // BLOCK, (w1 - 1) // BLOCK + 1):
                page, sub = int(cache["table"][i, blk // 4]), blk % 4
                sc = cache[which + "_scale"]
                place = range(blk * BLOCK, (blk + 1) * BLOCK)
                new = [p for p in place if w0 <= p < w1]
                kept = [p for p in place if p < lens[i] and not w0 <= p < w1]
                for g in range(hkv):
                    y = x[[p - w0 for p in new], g]
                    top = torch.where(torch.isfinite(y), y.abs(), torch.zeros(())).max()
                    scale = top * torch.tensor(1.0 / 127.0)
                    old = sc[page, g, sub].clone()
                    if kept:
                        scale = torch.maximum(scale, old)
                    if scale < 2.0 ** -100:
                        scale = torch.zeros(())
                    tile = cache[which][page, g, sub * BLOCK:(sub + 1) * BLOCK]
                    for p in kept:
                        if scale != old:
                            ratio = old / scale if scale > 0 else torch.zeros(())
                            tile[p % BLOCK] = torch.round(tile[p % BLOCK].float() * ratio).to(torch.int8)
                    inv = 1.0 / scale if scale > 0 else torch.zeros(())
                    z = y * inv
                    z = torch.where(torch.isnan(z), torch.zeros(()), torch.round(z)).clamp(-127, 127)
                    tile[[p % BLOCK for p in new]] = z.to(torch.int8)
                    sc[page, g, sub] = scale
                    out[which][[a + p - w0 for p in new], g] = (z * scale).to(k.dtype)
    return out


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, mask_id=-1):
    """(token, prob, kept ids) of one row, float64; the slowest way: sort, then
    add one token after the other."""
    z = np.asarray(logits, dtype=np.float64).copy()
    if mask_id >= 0:
        z[mask_id] = -np.inf
    z[np.isnan(z)] = -np.inf
    ids = [i for i in range(len(z)) if z[i] > -np.inf]
    if not ids:
        return -1, 0.0, []
    m = max(z[i] for i in ids)
    greedy = not temperature > 0
    t = 1.0 if greedy else float(temperature)
    w = {i: 1.0 if z[i] == m else (0.0 if m == np.inf else float(np.exp((z[i] - m) / t))) for i in ids}
    w = {i: (x if x >= 2.0 ** -45 else 0.0) for i, x in w.items()}
    ids.sort(key=lambda i: (-z[i], i))
    best = ids[0]
    if top_k > 0:
        ids = ids[:top_k]
    if not top_p >= 1:
        goal, before, kept = float(top_p) * sum(w[i] for i in ids), 0.0, []
        for i in ids:
            if kept and not before < goal:
                break
            kept.append(i)
            before += w[i]
        ids = kept
    if min_p > 0:
        ids = [i for i in ids if w[i] >= min(float(min_p), 1.0)]
    ids.sort()
    total = sum(w[i] for i in ids)
    if greedy:
        return best, w[best] / total, ids
    run, last = 0.0, -1
    for i in ids:
        run += w[i]
        if w[i] > 0:
            last = i
        if run > max(u, 0.0) * total:
            return i, w[i] / total, ids
    return last, w[last] / total, ids
