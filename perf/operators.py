"""Cases of the token-level attention operators: the norm and rotation of queries and keys,
the append to a paged key / value cache, and the attention of new tokens over that cache.

`listed()` gives the cases, `draw(rng)` one more of the same ranges, `prepare(case, seed)` a
case's inputs on the GPU, `run(state)` one pass of the operator, `work(case)` the bytes and
operations it cannot do without, and `exact(case, seed)` its outputs in 64 bits.  With `own`
false, `run` computes the plain form (elementary torch operations in FP32); with `own` true it
makes the library's calls.
"""

import random

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
K_SCALE, V_SCALE = 0.0175, 0.02  # static scales of an FP8 cache: normed keys and values reach 7 to 9


def _norm_rope(name, tokens, heads_q, heads_k, d, rot, interleaved, row_norm, fused):
    return dict(name=name, op="norm_rope", tokens=tokens, heads_q=heads_q, heads_k=heads_k, d=d, rot=rot,
                interleaved=interleaved, row_norm=row_norm, fused=fused)


def _append(name, seqs, q_min, q_max, kv_min, kv_max, heads_q, heads_k, d, page, fp8, interleaved, lens):
    return dict(name=name, op="append", seqs=seqs, q_min=q_min, q_max=q_max, kv_min=kv_min, kv_max=kv_max,
                heads_q=heads_q, heads_k=heads_k, d=d, page=page, fp8=fp8, interleaved=interleaved,
                heads_first=False, lens=lens)


def _attend(name, seqs, q_min, q_max, kv_min, kv_max, heads_q, heads_k, d, page, fp8, causal, window, heads_first,
            lens):
    return dict(name=name, op="attend", seqs=seqs, q_min=q_min, q_max=q_max, kv_min=kv_min, kv_max=kv_max,
                heads_q=heads_q, heads_k=heads_k, d=d, page=page, fp8=fp8, causal=causal, window=window,
                heads_first=heads_first, lens=lens)


def listed():
    return [
        # One generated token for each of five users, between the QKV projection and the attention: latency.
        _norm_rope("norm_rope_step", 5, 32, 8, 128, 128, False, False, True),
        # A prompt through a model with small heads and a rotation of half of each head, Q and K being
        # column slices of one fused projection.
        _norm_rope("norm_rope_partial", 4099, 16, 2, 64, 32, False, False, True),
        # Video self-attention: 32760 latent tokens, one norm over the whole row of 40 heads, rotated in
        # neighbouring pairs; the largest call of this operator.
        _norm_rope("norm_rope_video", 32760, 40, 40, 128, 128, True, True, False),
        # A generation step of 48 sequences: one token each into its page, with the queries rotated on the way.
        _append("append_step", 48, 1, 1, 16, 4096, 32, 8, 128, 16, False, False, 1),
        # Four chunks of prompts into an FP8 cache.
        _append("append_chunk_fp8", 4, 1500, 4096, 4096, 8192, 40, 8, 128, 64, True, True, 2),
        # One user, one token, a short context: the smallest attention, latency.
        _attend("decode_one", 1, 1, 1, 777, 777, 32, 8, 128, 16, False, True, 0, False, 3),
        # A generation step of 64 sequences of very different lengths.
        _attend("decode_ragged", 64, 1, 1, 1, 8192, 32, 8, 128, 16, False, True, 0, False, 4),
        # A generation step over long contexts in an FP8 cache.
        _attend("decode_long_fp8", 8, 1, 1, 30000, 65536, 64, 8, 128, 64, True, True, 0, False, 5),
        # Drafted tokens of 24 sequences checked at once, small heads, a sliding window, a cache laid out
        # head by head.
        _attend("draft_window", 24, 2, 6, 500, 6000, 16, 2, 64, 32, False, True, 1024, True, 6),
        # Chunked prefill: up to 2048 new tokens of four sequences over what the cache holds of each.
        _attend("chunk_ragged", 4, 500, 2048, 2048, 8192, 32, 8, 128, 16, False, True, 0, False, 7),
        # A whole prompt against an FP8 cache, five query heads for each key head.
        _attend("prompt_fp8", 1, 6001, 6001, 6001, 6001, 40, 8, 128, 64, True, True, 0, False, 8),
        # One latent frame of a video generated frame by frame: 1560 tokens over six frames, every key
        # visible, as many key heads as query heads.
        _attend("frame", 1, 1560, 1560, 9360, 9360, 40, 40, 128, 128, False, False, 0, False, 9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(2.0 ** rng.uniform(*[torch.tensor(float(v)).log2().item() for v in (lo, hi)])))))


def _drawn(rng):
    op = rng.choice(("norm_rope", "append", "attend", "attend"))
    d = rng.choice((64, 128))
    heads_k = rng.choice((1, 2, 4, 5, 8, 10))
    heads_q = heads_k * rng.choice((1, 2, 3, 4, 5, 7, 8))
    if op == "norm_rope":
        row = rng.random() < 0.3
        return _norm_rope("", _log(rng, 1, 32760), heads_q, heads_k, d, rng.choice((d, d, d // 2)), rng.random() < 0.5,
                          row, rng.random() < 0.5)
    seqs = _log(rng, 1, 64)
    page = rng.choice((8, 16, 24, 32, 64, 128))
    fp8 = rng.random() < 0.5
    step = rng.random() < 0.5
    q_max = rng.choice((1, 1, 2, 5, 8)) if step else _log(rng, 17, 4096)
    kv_max = max(q_max, _log(rng, 1, 65536 if step else 8192))
    q_min, kv_min = rng.randint(1, q_max), rng.randint(1, kv_max)
    lens = rng.randint(100, 1 << 30)
    if op == "append":
        return _append("", seqs, q_min, q_max, kv_min, kv_max, heads_q, heads_k, d, page, fp8, rng.random() < 0.5, lens)
    causal = rng.random() < 0.8
    window = _log(rng, 16, 4096) if causal and rng.random() < 0.3 else 0
    return _attend("", seqs, q_min, q_max, kv_min, kv_max, heads_q, heads_k, d, page, fp8, causal, window,
                   rng.random() < 0.4, lens)


def _cost(case):
    """What bounds a case's size: the operator's own work and the plain form's scores and gathered cache."""
    w = work(case)
    extra = 0
    if case["op"] != "norm_rope":
        q, kv = _lens(case)
        extra = len(q) * max(kv) * case["heads_k"] * case["d"] * 8
        extra += len(q) * max(q) * max(kv) * case["heads_q"] * 4 if case["op"] == "attend" else 0
    return max(w["bytes"], w["flops"] / 50, extra)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    c = _drawn(rng)
    while _cost(c) > most[c["op"]]:
        c = _drawn(rng)
    del c["name"]
    return c


def _lens(case):
    """New tokens and cached keys (the new ones among them) of each sequence: part of the case."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["seqs"])]
    kv = [r.randint(max(case["kv_min"], n), max(case["kv_max"], n)) for n in q]
    return q, kv


def _allowed(case):
    """Keys that the mask leaves to each sequence's rows, all rows together, and keys that any row reads."""
    q, kv = _lens(case)
    pairs, keys = 0, 0
    for n, L in zip(q, kv):
        if not case["causal"]:
            pairs, keys = pairs + n * L, keys + L
        elif not case["window"]:
            pairs, keys = pairs + n * (L - n) + n * (n + 1) // 2, keys + L
        else:
            w = case["window"]
            pairs += sum(min(w, L - n + i + 1) for i in range(n))
            keys += L - max(0, L - n + 1 - w)
    return pairs, keys


def work(case):
    d, hq, hk = case["d"], case["heads_q"], case["heads_k"]
    if case["op"] == "norm_rope":
        n = case["tokens"] * (hq + hk) * d
        table = case["tokens"] * case["rot"] * 4
        return {"bytes": 4 * n + table + case["tokens"] * 4, "flops": 8 * n}
    q, kv = _lens(case)
    T, size = sum(q), 1 if case["fp8"] else 2
    meta = 8 * len(q) + 4 * sum(-(-n // case["page"]) for n in kv)
    if case["op"] == "append":
        b = T * (hq * d * 4 + 2 * hk * d * (2 + size) + d * 4)
        return {"bytes": b + 8 * len(q) + 4 * T, "flops": 8 * T * (hq + hk) * d}
    pairs, keys = _allowed(case)
    return {"bytes": T * hq * d * 4 + keys * hk * d * 2 * size + meta, "flops": 4 * d * hq * pairs}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, tokens, width):
    """Projections as a norm meets them: a spread of channel scales."""
    return (_randn(g, tokens, width) * torch.exp(0.5 * _randn(g, width))).to(torch.bfloat16)


def _table(rows, rot):
    """cos and sin of position x 10000^(-2i / rot), formed in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _pool(g, case, fill):
    """A cache and its pages, dealt out in random order with some to spare."""
    q, kv = _lens(case)
    P, hk, d = case["page"], case["heads_k"], case["d"]
    need = [-(-n // P) for n in kv]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(q), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (pages, hk, P, d) if case["heads_first"] else (pages, P, hk, d)
    caches = []
    for scale in (K_SCALE, V_SCALE):
        c = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        if fill:
            for i in range(0, pages, 1 + (1 << 26) // (P * hk * d)):
                part = c[i:i + 1 + (1 << 26) // (P * hk * d)]
                part.copy_(_randn(g, *part.shape))
        if case["fp8"]:
            c = (c.float() / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        caches.append(c.transpose(1, 2) if case["heads_first"] else c)
    cu = torch.tensor([0] + [sum(q[:i + 1]) for i in range(len(q))], dtype=torch.int32, device="cuda")
    return dict(k_cache=caches[0], v_cache=caches[1], cu_q=cu, kv_len=torch.tensor(kv, dtype=torch.int32, device="cuda"),
                block_table=table, tokens=sum(q), q_max=max(q), kv_max=max(kv))


def prepare(case, seed):
    g = _gen(seed)
    d, hq, hk = case["d"], case["heads_q"], case["heads_k"]
    s = {"case": case}
    if case["op"] == "attend":
        s |= _pool(g, case, True)
        s["q"] = _randn(g, s["tokens"], hq * d).to(torch.bfloat16)
        return s
    row = case["op"] == "norm_rope" and case["row_norm"]
    rot = case["rot"] if case["op"] == "norm_rope" else d
    if case["op"] == "append":
        s |= _pool(g, case, False)
    T = s.get("tokens", case.get("tokens"))
    if case["op"] == "append" or case["fused"]:
        x = _activations(g, T, (hq + 2 * hk) * d)
        s["q"], s["k"], s["v"] = x[:, :hq * d], x[:, hq * d:(hq + hk) * d], x[:, (hq + hk) * d:]
    else:
        s["q"], s["k"] = _activations(g, T, hq * d), _activations(g, T, hk * d)
    for n, h in (("q", hq), ("k", hk)):
        s[n + "_weight"] = (1 + 0.2 * _randn(g, h * d if row else d)).to(torch.bfloat16)
    s["rot"] = rot
    if case["op"] == "norm_rope":
        s["table"] = _table(T + 64, rot)
        s["positions"] = torch.randint(0, 64, (1,), generator=g, device="cuda", dtype=torch.int32) + torch.arange(
            T, dtype=torch.int32, device="cuda")
    else:
        s["table"] = _table(s["kv_max"], rot)
    return s


def _norm_rotate(x, heads, weight, table, positions, rot, interleaved, row_norm):
    """w x / sqrt(mean(x^2) + eps) for each head or row, then the rotation of each head's first `rot` values."""
    T = x.shape[0]
    y = x.float().reshape(T, 1 if row_norm else heads, -1)
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.float()
    y = y.reshape(T, heads, -1)
    cs = table[positions.long()]
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    r = y[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, v], -1).reshape(T, heads, rot) if interleaved else torch.cat([u, v], -1)
    return torch.cat([r, y[..., rot:]], -1)


def _to_e4m3(y, scale):
    return (y * (1.0 / torch.tensor(scale, device=y.device))).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _places(s, case):
    """Sequence, position in it, page and slot in the page of each new token."""
    cu, t = s["cu_q"].long(), torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = t - cu[b] + s["kv_len"].long()[b] - (cu[b + 1] - cu[b])
    return pos, s["block_table"].long()[b, pos // case["page"]], pos % case["page"]


def _plain_append(s, case):
    pos, page, slot = _places(s, case)
    T, hk, d = s["tokens"], case["heads_k"], case["d"]
    il = case["interleaved"]
    k = _norm_rotate(s["k"], hk, s["k_weight"], s["table"], pos, d, il, False)
    v = s["v"].reshape(T, hk, d)
    s["k_cache"][page, slot] = _to_e4m3(k, K_SCALE) if case["fp8"] else k.to(torch.bfloat16)
    s["v_cache"][page, slot] = _to_e4m3(v.float(), V_SCALE) if case["fp8"] else v
    q = _norm_rotate(s["q"], case["heads_q"], s["q_weight"], s["table"], pos, d, il, False)
    return {"q": q.reshape(T, -1).to(torch.bfloat16), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s, case):
    B, mq, mk, P = case["seqs"], s["q_max"], s["kv_max"], case["page"]
    hq, hk, d = case["heads_q"], case["heads_k"], case["d"]
    ks, vs = (K_SCALE, V_SCALE) if case["fp8"] else (1.0, 1.0)
    j, i = torch.arange(mk, device="cuda"), torch.arange(mq, device="cuda")
    page = s["block_table"].long()[:, j // P].clamp(min=0)
    slot = (j % P).expand(B, mk)
    k = s["k_cache"][page, slot].float().transpose(1, 2) * ks  # [B, hk, mk, d]
    there = j < s["kv_len"][:, None]
    v = torch.where(there[:, None, :, None], s["v_cache"][page, slot].float().transpose(1, 2) * vs, 0.0)
    cu = s["cu_q"].long()
    n = cu[1:] - cu[:-1]
    inside = i < n[:, None]
    row = torch.where(inside, cu[:-1, None] + i, 0)
    q = s["q"][row].float().reshape(B, mq, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    pos = (s["kv_len"].long() - n)[:, None] + i
    ok = there[:, None, :].expand(B, mq, mk)
    if case["causal"]:
        ok = ok & (j <= pos[:, :, None])
        if case["window"]:
            ok = ok & (j > pos[:, :, None] - case["window"])
    ok = ok.repeat(1, hq // hk, 1)[:, None]
    x = torch.matmul(q.reshape(B, hk, -1, d), k.transpose(2, 3)) * d ** -0.5
    x = torch.where(ok, x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m.isinf(), 0.0, m))
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(total == 0, 1.0, total)
    o = o.reshape(B, hk, hq // hk, mq, d).permute(0, 3, 1, 2, 4).reshape(B, mq, hq * d)
    return o[inside].to(torch.bfloat16)


def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if case["op"] == "attend":
        return _plain_attend(s, case)
    if case["op"] == "append":
        return _plain_append(s, case)
    return {n: _norm_rotate(s[n], case["heads_" + n], s[n + "_weight"], s["table"], s["positions"], s["rot"],
                            case["interleaved"], case["row_norm"]).reshape(case["tokens"], -1).to(torch.bfloat16)
            for n in ("q", "k")}


def _own(s, case):
    from mxfp4_block_scaled_mxq_b200 import mxq

    if case["op"] == "norm_rope":
        q, k = mxq.qk_norm_rope(s["q"], s["k"], case["heads_q"], case["heads_k"], s["q_weight"], s["k_weight"], EPS,
                                mxq.MXQ_NORM_ROW if case["row_norm"] else mxq.MXQ_NORM_HEAD, s["table"],
                                s["positions"], mxq.MXQ_ROPE_PAIRS if case["interleaved"] else mxq.MXQ_ROPE_HALVES)
        return {"q": q, "k": k}
    cache = mxq.PagedKV(s["k_cache"], s["v_cache"], K_SCALE if case["fp8"] else 1.0, V_SCALE if case["fp8"] else 1.0)
    batch = mxq.PagedBatch(s["cu_q"], s["kv_len"], s["block_table"])
    if case["op"] == "append":
        q = mxq.kv_append(s["k"], s["v"], cache, batch, s["k_weight"], EPS, mxq.MXQ_NORM_HEAD, s["table"],
                          mxq.MXQ_ROPE_PAIRS if case["interleaved"] else mxq.MXQ_ROPE_HALVES,
                          q=s["q"], q_weight=s["q_weight"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return mxq.attention_paged(s["q"], case["heads_q"], cache, batch, causal=case["causal"], window=case["window"])


# ------------------------------------------------------------------ 64 bits, from the definitions
def _exact_head(x, weight, cos, sin, rot, interleaved, norm):
    """One head [T][d] of an operand: x / norm * weight as complex numbers times exp(i angle)."""
    y = x.double() / norm[:, None] * weight.double()
    re, im = (y[:, 0:rot:2], y[:, 1:rot:2]) if interleaved else (y[:, :rot // 2], y[:, rot // 2:rot])
    z = torch.complex(re, im) * torch.complex(cos, sin)
    out = y.clone()
    if interleaved:
        out[:, 0:rot:2], out[:, 1:rot:2] = z.real, z.imag
    else:
        out[:, :rot // 2], out[:, rot // 2:rot] = z.real, z.imag
    return out


def _exact_norm_rope(x, heads, weight, table, positions, rot, interleaved, row_norm):
    d = x.shape[1] // heads
    cs = table[positions.long()].double()
    cos, sin = cs[:, :rot // 2], cs[:, rot // 2:]
    whole = (x.double().square().sum(1) / x.shape[1] + EPS).sqrt() if row_norm else None
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for h in range(heads):
        part = x[:, h * d:(h + 1) * d]
        norm = whole if row_norm else (part.double().square().sum(1) / d + EPS).sqrt()
        w = weight[h * d:(h + 1) * d] if row_norm else weight
        out[:, h * d:(h + 1) * d] = _exact_head(part, w, cos, sin, rot, interleaved, norm)
    return out


def _exact_sequence(q, k, v, first, causal, window, hk):
    """softmax(q k^T / sqrt(d)) v of one sequence's rows, row i at position first + i; one key head at a time."""
    n, width = q.shape
    d = k.shape[2]
    group = width // d // hk
    out = torch.empty(n, width, dtype=torch.float64, device=q.device)
    far = torch.arange(k.shape[0], device=q.device)[None, :] - (first + torch.arange(n, device=q.device))[:, None]
    for h in range(hk * group):
        x = q[:, h * d:(h + 1) * d].double() @ k[:, h // group].double().T / d ** 0.5
        if causal:
            x.masked_fill_((far > 0) | ((far <= -window) if window else False), float("-inf"))
        out[:, h * d:(h + 1) * d] = torch.softmax(x, 1) @ v[:, h // group].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return {n: _exact_norm_rope(s[n], case["heads_" + n], s[n + "_weight"], s["table"], s["positions"], s["rot"],
                                    case["interleaved"], case["row_norm"]) for n in ("q", "k")}
    q, kv = _lens(case)
    ks, vs = (K_SCALE, V_SCALE) if case["fp8"] else (1.0, 1.0)
    if case["op"] == "attend":
        parts, at = [], 0
        for b, (n, L) in enumerate(zip(q, kv)):
            pages = s["block_table"][b, :-(-L // case["page"])].long()
            k, v = (s[c][pages].float().reshape(-1, case["heads_k"], case["d"])[:L].double() * w
                    for c, w in (("k_cache", ks), ("v_cache", vs)))
            parts.append(_exact_sequence(s["q"][at:at + n], k, v, L - n, case["causal"], case["window"], case["heads_k"]))
            at += n
        return torch.cat(parts)
    pos = torch.cat([torch.arange(L - n, L, device="cuda") for n, L in zip(q, kv)])
    b = torch.repeat_interleave(torch.arange(len(q), device="cuda"), torch.tensor(q, device="cuda"))
    page, slot = s["block_table"][b, pos // case["page"]].long(), pos % case["page"]
    new_q, new_k = (_exact_norm_rope(s[n], case["heads_" + n], s[n + "_weight"], s["table"], pos, case["d"],
                                     case["interleaved"], False) for n in ("q", "k"))
    out = {"q": new_q}
    for name, new, scale in (("k_cache", new_k, ks), ("v_cache", s["v"].double(), vs)):
        c = s[name].double()
        new = (new / scale).clamp(-E4M3_MAX, E4M3_MAX) if case["fp8"] else new
        c[page, slot] = new.reshape(len(pos), case["heads_k"], case["d"])
        out[name] = c
    return out
