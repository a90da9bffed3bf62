"""Norm and rotation of queries and keys (mxq_qk_norm_rope) and the append to a paged cache
(mxq_kv_append) against the formulas in 64 bits, and the whole step from projections to
attention as a model runs it."""

import pytest
import torch

import paged_ref as ref
from mxfp4_block_scaled_mxq_b200 import build, inputs, mxq
from parity import assert_status_clean

pytestmark = pytest.mark.gpu

SENTINEL = -12288.0  # exact in BF16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mxq.lib()
    yield
    assert_status_clean()


def _x(T, width, seed):
    return inputs.heavy_tailed_bf16(T, width, seed=seed, device="cuda")


def _w(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1 + 0.3 * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("row", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,d,rot", [(1, 1, 1, 64, 64), (3, 8, 2, 128, 128), (70, 40, 40, 128, 128),
                                           (33, 5, 1, 64, 32), (9, 3, 3, 80, 48), (17, 25, 5, 256, 64),
                                           (5, 64, 8, 128, 0), (4, 7, 2, 16, 16), (6, 2, 2, 96, 96)])
def test_norm_and_rotation(T, Hq, Hk, d, rot, row, pairs):
    q, k = _x(T, Hq * d, 1), _x(T, Hk * d, 2)
    qw, kw = _w(Hq * d if row else d, 3), _w(Hk * d if row else d, 4)
    table = mxq.rope_table(200, rot) if rot else None
    g = torch.Generator(device="cuda").manual_seed(T)
    pos = torch.randint(0, 200, (T,), generator=g, device="cuda", dtype=torch.int32)
    span, style = (mxq.MXQ_NORM_ROW if row else mxq.MXQ_NORM_HEAD), mxq.MXQ_ROPE_PAIRS if pairs else mxq.MXQ_ROPE_HALVES
    qo, ko = mxq.qk_norm_rope(q, k, Hq, Hk, qw, kw, 1e-6, span, table, pos, style)
    ref.assert_rounded(qo, *ref.norm_rope(q, Hq, qw, table, pos, 1e-6, row, pairs))
    ref.assert_rounded(ko, *ref.norm_rope(k, Hk, kw, table, pos, 1e-6, row, pairs))


def test_rotation_without_norm_and_norm_without_rotation():
    T, H, d = 50, 6, 128
    q, k = _x(T, H * d, 5), _x(T, H * d, 6)
    table = mxq.rope_table(T, d)
    pos = torch.arange(T, device="cuda")
    qo, ko = mxq.qk_norm_rope(q, k, H, H, table=table)  # positions 0, 1, 2, ...
    ref.assert_rounded(qo, *ref.norm_rope(q, H, None, table, pos, 0.0))
    ref.assert_rounded(ko, *ref.norm_rope(k, H, None, table, pos, 0.0))
    kw = _w(d, 7)
    qo, ko = mxq.qk_norm_rope(q, k, H, H, None, kw, 1e-5)
    assert torch.equal(qo, q)  # no weight, no table: the values as they are
    ref.assert_rounded(ko, *ref.norm_rope(k, H, kw, None, None, 1e-5))


def test_in_place_and_slices_of_a_fused_projection():
    """Q and K as column slices of one QKV matrix, in place; V and the rows' ends stay."""
    T, Hq, Hk, d = 77, 8, 2, 128
    x = _x(T, (Hq + 2 * Hk) * d + 8, 8)
    q, k = x[:, 8:8 + Hq * d], x[:, 8 + Hq * d:8 + (Hq + Hk) * d]
    qw, kw, table = _w(d, 9), _w(d, 10), mxq.rope_table(T, d)
    pos = torch.arange(T, device="cuda")
    before = x.clone()
    want_q, want_k = ref.norm_rope(q, Hq, qw, table, pos, 1e-6), ref.norm_rope(k, Hk, kw, table, pos, 1e-6)
    mxq.qk_norm_rope(q, k, Hq, Hk, qw, kw, table=table, q_out=q, k_out=k)
    ref.assert_rounded(q, *want_q)
    ref.assert_rounded(k, *want_k)
    assert torch.equal(x[:, :8], before[:, :8]) and torch.equal(x[:, 8 + (Hq + Hk) * d:], before[:, 8 + (Hq + Hk) * d:])


def test_rows_without_a_position_are_left():
    T, H, d = 12, 4, 64
    q, k = _x(T, H * d, 11), _x(T, H * d, 12)
    table = mxq.rope_table(30, d)
    pos = torch.tensor([0, 29, 30, -1, 5, 5, 1 << 30, -(1 << 31), 3, 2, 1, 29], dtype=torch.int32, device="cuda")
    qo, ko = (torch.full((T, H * d), SENTINEL, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mxq.qk_norm_rope(q, k, H, H, table=table, positions=pos, q_out=qo, k_out=ko)
    on = (pos >= 0) & (pos < 30)
    for got, x in ((qo, q), (ko, k)):
        assert (got[~on] == SENTINEL).all()
        w, m = ref.norm_rope(x[on], H, None, table, pos[on], 0.0)
        ref.assert_rounded(got[on], w, m)


def test_zero_rows_and_far_positions():
    """A zero vector stays zero (eps), and a table whose angles were formed in 64 bits holds at
    position 10^6."""
    d = 128
    q = torch.zeros(2, d, dtype=torch.bfloat16, device="cuda")
    q[1] = 1.0
    table = mxq.rope_table(torch.tensor([0, 10 ** 6]), d)
    qo, ko = mxq.qk_norm_rope(q, q.clone(), 1, 1, _w(d, 1), None, 1e-6, table=table)
    assert (qo[0] == 0).all()
    inv = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d) * 1e6
    want = torch.cat([inv.cos() - inv.sin(), inv.cos() + inv.sin()])
    # table entries are within 2^-25 of the exact ones, plus those of the FP64 angle (1e6 x 2^-53)
    assert ((ko[1].double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -17 * 2).all()


def _cache(pages, page, Hk, d, fp8, heads_first=False):
    shape = (pages, Hk, page, d) if heads_first else (pages, page, Hk, d)
    kv = []
    for _ in range(2):
        c = torch.full(shape, SENTINEL if not fp8 else -96.0, device="cuda")
        c = c.to(torch.float8_e4m3fn if fp8 else torch.bfloat16)
        kv.append(c.transpose(1, 2) if heads_first else c)
    return mxq.PagedKV(*kv, *((0.03, 0.05) if fp8 else (1.0, 1.0)))


def _batch(q_lens, kv_lens, page, seed, max_pages=None):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in kv_lens]
    order = torch.randperm(sum(need) + 2, generator=g).to(torch.int32)
    table = torch.full((len(q_lens), max_pages or max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cu = torch.tensor([0, *torch.tensor(q_lens).cumsum(0).tolist()], dtype=torch.int32)
    batch = mxq.PagedBatch(cu.cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda(), table.cuda())
    places = [(int(table[b, p // page]), p % page, p) for b, (n, L) in enumerate(zip(q_lens, kv_lens))
              for p in range(L - n, L)]
    return batch, sum(need) + 2, places


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hk,d,page,pairs", [
    ([1, 1, 1], [1, 17, 300], 8, 2, 128, 16, False), ([5, 0, 64, 1], [9, 40, 64, 33], 4, 4, 64, 8, True),
    ([130], [200], 40, 8, 128, 24, True), ([1] * 70, list(range(1, 71)), 5, 1, 80, 32, False)])
def test_append(q_lens, kv_lens, Hq, Hk, d, page, pairs, heads_first, fp8):
    batch, pages, places = _batch(q_lens, kv_lens, page, 3)
    cache = _cache(pages, page, Hk, d, fp8, heads_first)
    T, pad = sum(q_lens), 4
    x = _x(T + pad, (Hq + 2 * Hk) * d, 21)
    q, k, v = x[:, :Hq * d], x[:, Hq * d:(Hq + Hk) * d], x[:, (Hq + Hk) * d:]
    qw, kw, table = _w(d, 22), _w(d, 23), mxq.rope_table(max(kv_lens), d)
    style = mxq.MXQ_ROPE_PAIRS if pairs else mxq.MXQ_ROPE_HALVES
    qo = torch.full((T + pad, Hq * d), SENTINEL, dtype=torch.bfloat16, device="cuda")
    before = [c.float().clone() for c in (cache.k, cache.v)]
    mxq.kv_append(k, v, cache, batch, kw, 1e-6, table=table, style=style, q=q, q_weight=qw, q_out=qo)
    pg, slot, pos = (torch.tensor(z, device="cuda") for z in zip(*places))
    ref.assert_rounded(qo[:T], *ref.norm_rope(q[:T], Hq, qw, table, pos, 1e-6, False, pairs))
    assert (qo[T:] == SENTINEL).all()
    want_k, mag_k = ref.norm_rope(k[:T], Hk, kw, table, pos, 1e-6, False, pairs)
    got_k, got_v = cache.k.view(torch.uint8)[pg, slot].view(cache.k.dtype) if fp8 else cache.k[pg, slot], None
    ref.assert_rounded(got_k.reshape(T, -1), want_k, mag_k, cache.args.k_scale)
    if fp8:
        inv = 1.0 / torch.tensor(cache.args.v_scale, dtype=torch.float32, device="cuda")
        want_v = (v[:T].float() * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        got_v = cache.v.view(torch.uint8)[pg, slot]
    else:
        want_v, got_v = v[:T], cache.v[pg, slot]
    assert torch.equal(got_v.reshape(T, -1), want_v.contiguous().reshape(T, -1))  # values are not computed on
    for c, old in zip((cache.k, cache.v), before):  # every other place keeps its contents
        new = c.float().clone()
        new[pg, slot] = old[pg, slot]
        assert torch.equal(new, old)
    # without queries the cache is the same
    again = _cache(pages, page, Hk, d, fp8, heads_first)
    assert mxq.kv_append(k, v, again, batch, kw, 1e-6, table=table, style=style) is None
    assert torch.equal(again.k.float(), cache.k.float()) and torch.equal(again.v.float(), cache.v.float())


def test_append_of_rows_norm():
    """One norm over the whole row of heads, queries and keys apart."""
    batch, pages, places = _batch([40], [100], 16, 4)
    cache = _cache(pages, 16, 8, 128, False)
    q, k, v = _x(40, 40 * 128, 24), _x(40, 8 * 128, 25), _x(40, 8 * 128, 26)
    qw, kw, table = _w(40 * 128, 27), _w(8 * 128, 28), mxq.rope_table(100, 128)
    qo = mxq.kv_append(k, v, cache, batch, kw, 1e-6, mxq.MXQ_NORM_ROW, table, q=q, q_weight=qw)
    pg, slot, pos = (torch.tensor(z, device="cuda") for z in zip(*places))
    ref.assert_rounded(qo, *ref.norm_rope(q, 40, qw, table, pos, 1e-6, True))
    ref.assert_rounded(cache.k[pg, slot].reshape(40, -1), *ref.norm_rope(k, 8, kw, table, pos, 1e-6, True))


def test_append_skips_what_has_no_place():
    """Missing pages (the queries are still written), positions before 0, beyond the block table
    and beyond the rotation table: the cache and the queries' rows keep their contents."""
    page, Hk, d = 8, 2, 64
    table = mxq.rope_table(20, d)
    cu = torch.tensor([0, 3, 6, 9, 12], dtype=torch.int32, device="cuda")
    kv = torch.tensor([2, 21, 10, 26], dtype=torch.int32, device="cuda")
    bt = torch.tensor([[0, 1, 2], [3, 4, 5], [6, -1, 7], [8, 99, 9]], dtype=torch.int32, device="cuda")
    cache = _cache(10, page, Hk, d, False)
    k, v, q = _x(13, Hk * d, 30), _x(13, Hk * d, 31), _x(13, 4 * d, 32)
    qo = torch.full((13, 4 * d), SENTINEL, dtype=torch.bfloat16, device="cuda")
    mxq.kv_append(k, v, cache, mxq.PagedBatch(cu, kv, bt), table=table, q=q, q_out=qo)
    # positions: -1 0 1 | 18 19 20 | 7 8 9 | 23 24 25
    place = {1: (0, 0), 2: (0, 1), 3: (5, 2), 4: (5, 3), 6: (6, 7)}
    written = [1, 2, 3, 4, 6, 7, 8]
    pos = {1: 0, 2: 1, 3: 18, 4: 19, 6: 7, 7: 8, 8: 9}
    for r in range(13):
        if r in written:
            ref.assert_rounded(qo[r:r + 1], *ref.norm_rope(q[r:r + 1], 4, None, table, torch.tensor([pos[r]]).cuda(), 0.0))
        else:
            assert (qo[r] == SENTINEL).all()
    kc, vc = cache.k.clone(), cache.v.clone()
    for r, (g, s) in place.items():
        ref.assert_rounded(kc[g, s].reshape(1, -1), *ref.norm_rope(k[r:r + 1], Hk, None, table, torch.tensor([pos[r]]).cuda(), 0.0))
        assert torch.equal(vc[g, s].reshape(-1), v[r])
        kc[g, s] = vc[g, s] = SENTINEL
    assert (kc == SENTINEL).all() and (vc == SENTINEL).all()


def test_append_into_the_last_pages_of_a_cache_beyond_32_bits():
    page, Hk, d = 16, 8, 128
    pages = (1 << 31) // (page * Hk * d) + 5
    k_cache, v_cache = (torch.empty(pages, page, Hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = _x(20, Hk * d, 33), _x(20, Hk * d, 34)
    batch = mxq.PagedBatch(torch.tensor([0, 20], dtype=torch.int32, device="cuda"),
                           torch.tensor([20], dtype=torch.int32, device="cuda"),
                           torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda"))
    mxq.kv_append(k, v, mxq.PagedKV(k_cache, v_cache), batch)
    assert torch.equal(k_cache[pages - 1].reshape(16, -1), k[:16]) and torch.equal(v_cache[pages - 3][:4].reshape(4, -1), v[16:])


@pytest.mark.parametrize("fp8", [False, True])
def test_a_model_step_from_projections_to_the_output(fp8):
    """As a model runs them: a prompt of each sequence, then generated tokens, through the W4A4
    QKV projection, the append with norm and rotation, and the attention; the generation step
    captured into a CUDA graph and replayed while the lengths grow.  Each step's output is
    checked against the formula on the cache as it then is."""
    Hq, Hk, d, K, page = 8, 2, 128, 512, 16
    width = (Hq + 2 * Hk) * d
    wc, wsf = mxq.pack_weight(inputs.normal_bf16(width, K, 0.05, seed=40).cuda())
    qw, kw, table = _w(d, 41), _w(d, 42), mxq.rope_table(256, d)
    fmt = mxq.MXQ_KV_FP8_E4M3 if fp8 else mxq.MXQ_KV_BF16
    cache = mxq.paged_kv(40, page, Hk, d, fmt, *((0.03, 0.05) if fp8 else (1.0, 1.0)))
    for c in (cache.k, cache.v):
        c.view(torch.uint8).fill_(0x7F if fp8 else 0xFF)  # NaN
    bt = torch.randperm(40, generator=torch.Generator().manual_seed(1))[:30].reshape(3, 10).to(torch.int32).cuda()
    kv_len = torch.zeros(3, dtype=torch.int32, device="cuda")

    def step(x, batch):
        qkv = mxq.linear_w4a4(x, wc, wsf, width)
        q, k, v = qkv[:, :Hq * d], qkv[:, Hq * d:(Hq + Hk) * d], qkv[:, (Hq + Hk) * d:]
        q = mxq.kv_append(k, v, cache, batch, kw, table=table, q=q, q_weight=qw)
        return q, mxq.attention_paged(q, Hq, cache, batch)

    def check(q, o, batch):
        want, mags, owned = ref.attention(q, Hq, cache.k, cache.v, batch.cu_q, batch.kv_len, batch.block_table,
                                          k_scale=cache.args.k_scale, v_scale=cache.args.v_scale)
        ref.assert_attention(o, want, mags, owned)

    lens = [100, 33, 7]
    kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
    prompt = mxq.PagedBatch(torch.tensor([0, 100, 133, 140], dtype=torch.int32, device="cuda"), kv_len, bt)
    x = inputs.normal_bf16(140, K, 1.0, seed=43).cuda()
    check(*step(x, prompt), prompt)

    batch = mxq.PagedBatch(torch.arange(4, dtype=torch.int32, device="cuda"), kv_len, bt)
    x1 = inputs.normal_bf16(3, K, 1.0, seed=44).cuda()
    kv_len += 1
    check(*step(x1, batch), batch)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        kv_len += 1
        q, o = step(x1, batch)
    for i in range(20):
        x1.copy_(inputs.normal_bf16(3, K, 1.0, seed=50 + i))
        g.replay()
        if i % 6 == 0:
            check(q, o, batch)
    torch.cuda.synchronize()
    assert kv_len.tolist() == [n + 21 for n in lens]


def test_norm_rope_before_the_mxfp4_attention():
    """The norm and rotation feed the MXFP4 attention of one sequence like any Q and K."""
    T, H, d = 300, 2, 128
    q, k, v = _x(T, H * d, 60), _x(T, H * d, 61), inputs.normal_bf16(T, H * d, 1.0, seed=62).cuda()
    table, w = mxq.rope_table(T, d), _w(d, 63)
    qo, ko = mxq.qk_norm_rope(q, k, H, H, w, w, table=table, style=mxq.MXQ_ROPE_PAIRS)
    pos = torch.arange(T, device="cuda")
    rq, rk = (ref.norm_rope(x, H, w, table, pos, 1e-6, False, True) for x in (q, k))
    ref.assert_rounded(qo, *rq)
    ref.assert_rounded(ko, *rk)
    a = mxq.attention_mxfp4(qo, ko, v, H)
    b = mxq.attention_mxfp4(qo.clone(), ko.clone(), v, H)
    assert torch.equal(a, b) and torch.isfinite(a).all()


@pytest.mark.parametrize("T", [1, 500])
def test_streams_and_graphs(T):
    q, k = _x(T, 8 * 128, 70), _x(T, 2 * 128, 71)
    w, table = _w(128, 72), mxq.rope_table(T, 128)
    want = mxq.qk_norm_rope(q, k, 8, 2, w, w, table=table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mxq.qk_norm_rope(q, k, 8, 2, w, w, table=table, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.zeros_like(x) for x in want]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mxq.qk_norm_rope(q, k, 8, 2, w, w, table=table, q_out=outs[0], k_out=outs[1])
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("row", [False, True])
@pytest.mark.parametrize("Hq,Hk,d", [(512, 512, 128), (256, 40, 256), (1024, 3, 64), (455, 455, 144)])
def test_rows_wider_than_a_block_holds(Hq, Hk, d, row, pairs):
    """Rows of up to 2^16 values a side are divided over blocks, by heads or (one norm over the
    row) by operands; in the append queries, keys and values may lie in one block or not."""
    T = 5
    q, k, v = _x(T, Hq * d, 80), _x(T, Hk * d, 81), _x(T, Hk * d, 82)
    qw, kw = _w(Hq * d if row else d, 83), _w(Hk * d if row else d, 84)
    table = mxq.rope_table(50, d)
    span, style = (mxq.MXQ_NORM_ROW if row else mxq.MXQ_NORM_HEAD), mxq.MXQ_ROPE_PAIRS if pairs else mxq.MXQ_ROPE_HALVES
    batch, pages, places = _batch([3, 2], [30, 9], 8, 5)
    pg, slot, pos = (torch.tensor(z, device="cuda") for z in zip(*places))
    want_q = ref.norm_rope(q, Hq, qw, table, pos, 1e-6, row, pairs)
    want_k = ref.norm_rope(k, Hk, kw, table, pos, 1e-6, row, pairs)
    qo, ko = mxq.qk_norm_rope(q, k, Hq, Hk, qw, kw, 1e-6, span, table, pos.to(torch.int32), style)
    ref.assert_rounded(qo, *want_q)
    ref.assert_rounded(ko, *want_k)
    for queries in (q, None):
        cache = _cache(pages, 8, Hk, d, False)
        got = mxq.kv_append(k, v, cache, batch, kw, 1e-6, span, table, style, queries, qw if queries is not None else None)
        if queries is not None:
            ref.assert_rounded(got, *want_q)
        ref.assert_rounded(cache.k[pg, slot].reshape(T, -1), *want_k)
        assert torch.equal(cache.v[pg, slot].reshape(T, -1), v)


def test_more_tokens_than_a_block_looks_up_at_once():
    """A block takes every so-many-th token and looks 32 up at a time: several such rounds."""
    T, d, page = 40003, 64, 16
    q, k, v = _x(T, 2 * d, 85), _x(T, d, 86), _x(T, d, 87)
    w, table = _w(d, 88), mxq.rope_table(T, d)
    lens = [T - 40 * 700, *[40] * 700]
    batch, pages, places = _batch(lens, lens, page, 6)
    pg, slot, pos = (torch.tensor(z, device="cuda") for z in zip(*places))
    qo, ko = mxq.qk_norm_rope(q, k, 2, 1, w, w, table=table, positions=pos.to(torch.int32))
    want_q, want_k = ref.norm_rope(q, 2, w, table, pos, 1e-6), ref.norm_rope(k, 1, w, table, pos, 1e-6)
    ref.assert_rounded(qo, *want_q)
    ref.assert_rounded(ko, *want_k)
    cache = mxq.paged_kv(pages, page, 1, d)
    assert torch.equal(mxq.kv_append(k, v, cache, batch, w, table=table, q=q, q_weight=w), qo)
    assert torch.equal(cache.k[pg, slot].reshape(T, -1), ko) and torch.equal(cache.v[pg, slot].reshape(T, -1), v)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_stay_in_their_head(bad):
    """An infinity or NaN spoils its own head's norm; every other head is as without it."""
    T, H, d = 4, 6, 128
    q, k = _x(T, H * d, 89), _x(T, H * d, 90)
    w, table = _w(d, 91), mxq.rope_table(T, d)
    want_q, want_k = mxq.qk_norm_rope(q, k, H, H, w, w, table=table)
    q[2, 3 * d + 7] = bad
    qo, ko = mxq.qk_norm_rope(q, k, H, H, w, w, table=table)
    assert torch.isnan(qo[2, 3 * d + 7]) and torch.equal(ko, want_k)
    qo[2, 3 * d:4 * d] = want_q[2, 3 * d:4 * d]
    assert torch.equal(qo, want_q)


def test_e4m3_append_at_the_ends_of_the_type():
    """Values and keys beyond the type's range saturate, NaN stays NaN, the smallest round to even."""
    d, page = 64, 8
    x = torch.zeros(6, d, device="cuda")
    x[0], x[1], x[2], x[3] = 1e6, -1e6, float("nan"), float("inf")
    x[4, :4] = torch.tensor([2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, -2.0 ** -11])
    x[5] = torch.linspace(-460, 460, d)
    x = x.to(torch.bfloat16)
    cache = mxq.PagedKV(*(torch.zeros(1, page, 1, d, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)))
    z = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    mxq.kv_append(x, x, cache, mxq.PagedBatch(z, z[1:], torch.zeros(1, 1, dtype=torch.int32, device="cuda")))
    want = x.float().clamp(-448, 448).to(torch.float8_e4m3fn)
    for c in (cache.k, cache.v):
        got = c[0, :6, 0].float()
        assert torch.equal(torch.isnan(got), torch.isnan(x)) and torch.equal(torch.nan_to_num(got), torch.nan_to_num(want.float()))


def test_append_with_queries_in_place():
    """Q, K and V as slices of one projection, the queries rotated where they are."""
    batch, pages, places = _batch([30, 1], [60, 33], 16, 7)
    Hq, Hk, d = 8, 2, 128
    x = _x(31, (Hq + 2 * Hk) * d, 92)
    before = x.clone()
    q, k, v = x[:, :Hq * d], x[:, Hq * d:(Hq + Hk) * d], x[:, (Hq + Hk) * d:]
    qw, kw, table = _w(d, 93), _w(d, 94), mxq.rope_table(64, d)
    pos = torch.tensor([p for _, _, p in places], device="cuda")
    want = ref.norm_rope(q, Hq, qw, table, pos, 1e-6)
    cache = _cache(pages, 16, Hk, d, False)
    assert mxq.kv_append(k, v, cache, batch, kw, table=table, q=q, q_weight=qw, q_out=q) is q
    ref.assert_rounded(q, *want)
    assert torch.equal(x[:, Hq * d:], before[:, Hq * d:])
