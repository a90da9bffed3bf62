"""Plain 64-bit references of the norm and rotation, the cache append and the paged attention,
and the tolerances of their tests (derived in the comments, none measured)."""

from __future__ import annotations

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}


def norm_rope(x, heads, weight, table, positions, eps, row=False, pairs=False):
    """([T][heads * d] result, magnitudes): norm and rotation in FP64; the magnitude of a value is
    the sum of the absolute values of its rotated pair, to which FP32 rounding errors are relative."""
    T, width = x.shape
    d = width // heads
    y = x.double().reshape(T, heads, d)
    if weight is not None:
        ss = y.square().mean((1, 2) if row else 2, keepdim=True)
        y = y / (ss + eps).sqrt() * (weight.double().reshape(heads, d) if row else weight.double())
    mag = y.abs()
    if table is not None:
        rot = table.shape[1]
        cs = table[positions.long()].double()[:, None, :]
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
        out, mag = y.clone(), mag.clone()
        cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
        out[..., a] = y[..., a] * cos - y[..., b] * sin
        out[..., b] = y[..., b] * cos + y[..., a] * sin
        mag[..., a] = mag[..., b] = y[..., a].abs() + y[..., b].abs()
        y = out
    return y.reshape(T, width), mag.reshape(T, width)


def assert_rounded(got, want, mag, scale=1.0):
    """got (BF16, or E4M3 with its scale) is `want` rounded once from an FP32 computation.

    FP32: the sum of squares is off by at most 64 x 2^-24 relative (a term passes through 6 roundings
    in its lane's head, one for each of up to 33 heads of the lane, and 9 in the tree over lanes and
    warps), half of that after the square root; the root (2 units in the last place), two products
    and the rotation's three operations add 9 x 2^-24: under 2^-17 of the pair's magnitude,
    rotated by |cos|, |sin| <= 1.  Then half a step of the result's type (BF16 2^-8
    relative; E4M3 2^-4 relative, 2^-10 absolute below its normal range)."""
    want, mag = want / scale, mag / scale
    g = got.double()
    if got.dtype == torch.float8_e4m3fn:
        want = want.clamp(-448.0, 448.0)
        step = (want.abs() * 2.0 ** -4).clamp(min=2.0 ** -10)
    else:
        step = want.abs() * 2.0 ** -8
    tol = step + 2.0 ** -17 * mag * (1 + 2.0 ** -4)
    assert torch.isfinite(g).all()
    bad = (g - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((g - want).abs() - tol).max()))


def pages_of(batch_table, b, n, page):
    return [int(x) for x in batch_table[b, :-(-n // page)]] if n > 0 else []


def attention(q, Hq, k_cache, v_cache, cu_q, kv_len, block_table, causal=True, window=0, scale=None, k_scale=1.0,
              v_scale=1.0):
    """FP64 rows (T, Hq * d), the weighted sums of |V| that the rounding of the weights is relative
    to, and which rows belong to a sequence.  Missing pages' keys are masked."""
    T, width = q.shape
    d = width // Hq
    P, Hk = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hk
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device=q.device)
    mags, owned = torch.zeros_like(out), torch.zeros(T, dtype=torch.bool, device=q.device)
    cu, lens = cu_q.tolist(), kv_len.tolist()
    num_pages = k_cache.shape[0]
    for b, L in enumerate(lens):
        r0, r1 = cu[b], cu[b + 1]
        n = r1 - r0
        owned[r0:r1] = True
        L = min(max(L, 0), block_table.shape[1] * P)
        if n == 0 or L == 0:
            continue
        entries = block_table[b, :-(-L // P)].long()
        there = ((entries >= 0) & (entries < num_pages)).repeat_interleave(P)[:L]
        pg = entries.clamp(0, num_pages - 1)
        k = k_cache[pg].float().double().reshape(-1, Hk, d)[:L] * k_scale
        v = v_cache[pg].float().double().reshape(-1, Hk, d)[:L] * v_scale
        v = torch.where(there[:, None, None], v, 0.0)
        pos = L - n + torch.arange(n, device=q.device)[:, None]
        j = torch.arange(L, device=q.device)[None, :]
        ok = there[None, :].expand(n, L)
        if causal:
            ok = ok & (j <= pos)
            if window:
                ok = ok & (j > pos - window)
        for h in range(Hq):
            s = q[r0:r1, h * d:(h + 1) * d].double() @ k[:, h // G].T * scale
            s = torch.where(ok, s, float("-inf"))
            m = s.amax(1, keepdim=True)
            e = torch.exp(s - torch.where(m.isinf(), 0.0, m))
            e = torch.where(ok, e, 0.0)
            total = e.sum(1, keepdim=True)
            w = e / torch.where(total == 0, 1.0, total)
            out[r0:r1, h] = w @ v[:, h // G]
            mags[r0:r1, h] = w @ v[:, h // G].abs()
    return out.reshape(T, width), mags.reshape(T, width), owned


def assert_attention(got, want, mags, owned):
    """Each weight is rounded to BF16 (2^-8 relative, at most) or FP16, the result to BF16 (2^-8).
    FP32 scores: the d products of a score add up with d x 2^-24 x sum |q k| x scale at most, under
    2^-10 for the unit-variance operands of these tests (sum |q k| scale < 64 for d = 128),
    which changes every weight by less than 2^-10 relative and the sums by as much."""
    g = got.double()
    tol = (2.0 ** -8 + 2.0 ** -9) * mags + 2.0 ** -8 * want.abs() + 1e-30
    err = (g - want).abs()
    bad = (err > tol) | ~torch.isfinite(g)
    bad = bad[owned]
    assert not bad.any(), (int(bad.sum()), bad.numel(), float((err / tol)[owned].max()))
