"""Paged attention (mxq_attention_paged) against the formula in 64 bits: few rows and many,
grouped heads, both cache types, page sizes and orders, causal, windowed and open masks, rows and
sequences without keys, missing pages, garbage in unused places, and rows of no sequence."""

import pytest
import torch

import paged_ref as ref
from mxfp4_block_scaled_mxq_b200 import build, mxq
from parity import assert_status_clean

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mxq.lib()
    yield
    assert_status_clean()


SENTINEL = -12288.0  # exact in BF16


def make(q_lens, kv_lens, Hq, Hk, d, page, fp8=False, heads_first=False, seed=0, pad=0, spare=2, fill=float("nan"),
         max_pages=None):
    """Inputs whose unused cache places hold `fill`; pages dealt out in random order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(q_lens)
    need = [-(-n // page) for n in kv_lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max_pages or max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    shape = (pages, Hk, page, d) if heads_first else (pages, page, Hk, d)
    caches = []
    scales = (0.02, 0.03) if fp8 else (1.0, 1.0)
    for sc in scales:
        c = torch.randn(shape, generator=g, device="cuda")
        c = (c / sc).clamp(-448, 448).to(torch.float8_e4m3fn) if fp8 else c.to(torch.bfloat16)
        caches.append(c.transpose(1, 2) if heads_first else c)
    at = 0
    used = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        if n:
            flat = torch.arange(n * page, device="cuda").reshape(n, page) < kv_lens[b]
            used[order[at:at + n].long()] = flat
        at += n
    for c in caches:
        raw = c.view(torch.uint8) if fp8 else c
        raw.copy_(torch.where(used[:, :, None, None], raw, torch.tensor(0x7F if fp8 else fill, dtype=raw.dtype,
                                                                         device="cuda")))
    cu = torch.tensor([0, *torch.tensor(q_lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    T = sum(q_lens) + pad
    q = torch.randn(T, Hq * d, generator=g, device="cuda").to(torch.bfloat16)
    return dict(q=q, Hq=Hq, k_cache=caches[0], v_cache=caches[1], cu_q=cu,
                kv_len=torch.tensor(kv_lens, dtype=torch.int32, device="cuda"), block_table=table, k_scale=scales[0],
                v_scale=scales[1])


def call(s, out=None, **kw):
    cache = mxq.PagedKV(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    batch = mxq.PagedBatch(s["cu_q"], s["kv_len"], s["block_table"])
    return mxq.attention_paged(s["q"], s["Hq"], cache, batch, out=out, **kw)


def check(s, **kw):
    out = torch.full(s["q"].shape, SENTINEL, dtype=torch.bfloat16, device="cuda")
    call(s, out=out, **kw)
    want, mags, owned = ref.attention(s["q"], s["Hq"], s["k_cache"], s["v_cache"], s["cu_q"], s["kv_len"],
                                      s["block_table"], k_scale=s["k_scale"], v_scale=s["v_scale"], **kw)
    ref.assert_attention(out, want, mags, owned)
    assert (out[~owned] == SENTINEL).all()
    return out, want


HEADS = [(8, 8), (8, 2), (5, 1), (16, 1), (21, 3), (40, 1)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hk", HEADS)
def test_single_tokens(Hq, Hk, d, fp8):
    """One token each: lengths of one, around the key tiles, and some hundreds."""
    kv = [1, 2, 31, 32, 33, 63, 64, 65, 100, 255, 256, 257, 700]
    check(make([1] * len(kv), kv, Hq, Hk, d, 16, fp8, seed=Hq))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [8, 16, 24, 40, 64, 128, 256])
@pytest.mark.parametrize("heads_first", [False, True])
def test_page_sizes_and_orders(page, fp8, heads_first):
    check(make([1, 3, 2], [3 * page + 5, 700, page], 8, 2, 128, page, fp8, heads_first, seed=page))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 40), (True, 5000), (False, 0)])
def test_masks_over_chunks(causal, window, d, fp8):
    """Chunks of a few to some hundreds of tokens behind cached ones, and without."""
    check(make([1, 5, 17, 130, 300], [400, 5, 200, 131, 300], 8, 2, d, 16, fp8, seed=3), causal=causal, window=window)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hk,d", [(4, 4, 128), (8, 2, 64), (10, 2, 128), (16, 1, 128), (7, 1, 64), (40, 8, 128)])
def test_long_chunks(Hq, Hk, d, fp8):
    """Many row tiles of every group size, beside single tokens and a sequence without new ones."""
    check(make([333, 1, 0, 257, 64], [1000, 500, 77, 257, 640], Hq, Hk, d, 32, fp8, seed=Hq + d))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_lens", [[1, 0, 2, 1], [200, 0, 90, 1]])
def test_rows_without_keys_are_zero(q_lens, fp8):
    """No cached key at all; more new tokens than cached keys (the first rows' positions are
    negative); a sequence without rows."""
    s = make(q_lens, [0, 50, 1, 64], 8, 2, 128, 16, fp8, seed=5, pad=3)
    out, _ = check(s)
    n0, n1 = q_lens[0], q_lens[0] + q_lens[1]
    assert (out[:n0] == 0).all()
    assert (out[n1:n1 + q_lens[2] - 1] == 0).all()


@pytest.mark.parametrize("q_lens", [[2, 1], [150, 129]])
def test_missing_pages_are_not_attended(q_lens):
    s = make(q_lens, [300, 300], 8, 2, 128, 16, seed=6)
    s["block_table"][0, 3] = -1
    s["block_table"][0, 7:9] = s["k_cache"].shape[0]
    s["block_table"][0, 18] = 1 << 30
    s["block_table"][1, :] = -5
    out, _ = check(s)
    assert (out[q_lens[0]:] == 0).all()
    s["block_table"][0, 5] = -1
    check(s, causal=False)
    check(s, window=64)


@pytest.mark.parametrize("q_lens", [[1, 1], [140, 3]])
def test_lengths_beyond_the_table_are_clamped(q_lens):
    s = make(q_lens, [160, 160], 4, 2, 128, 16, seed=7)
    want = call(s)
    s["kv_len"][:] = 100000
    assert torch.equal(call(s), want)
    s["kv_len"][0] = -7
    # where a unit is split depends on all lengths, so the other sequence is equal up to the
    # rounding of the joined parts: held to the formula
    out, _ = check(s)
    assert (out[:q_lens[0]] == 0).all()


@pytest.mark.parametrize("q_lens", [[1, 4], [150, 40]])
def test_garbage_behind_a_window_does_not_leak(q_lens):
    """Keys and values that every row's window has left may be anything."""
    s = make(q_lens, [400, 300], 4, 2, 128, 16, seed=8)
    first = s["block_table"][0, :5].long()  # positions 0..79: positions - window of all rows of sequence 0 are later
    s["k_cache"][first] = float("inf")
    s["v_cache"][first] = float("nan")
    window = 100 if q_lens[0] == 1 else 150
    clean = {**s, "k_cache": torch.nan_to_num(s["k_cache"], 0, 0, 0), "v_cache": torch.nan_to_num(s["v_cache"], 0, 0, 0)}
    out = call(s, window=window)
    assert torch.isfinite(out).all() and torch.equal(out, call(clean, window=window))


@pytest.mark.parametrize("q_lens,pad", [([1, 1, 1], 5), ([100, 30], 200)])
def test_rows_of_no_sequence_keep_their_contents(q_lens, pad):
    check(make(q_lens, [90 + 100 * i + q_lens[i] for i in range(len(q_lens))], 8, 4, 64, 16, seed=9, pad=pad))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 200])
def test_long_context_split_over_many_ctas(n, fp8):
    """One sequence, one key head: every CTA holds a part of the same unit."""
    check(make([n], [20011], 4, 1, 128, 64, fp8, seed=10))


def test_many_short_sequences():
    """More sequences than a block has threads, lengths 0 to 40."""
    B = 1500
    q = [(i * 7) % 3 for i in range(B)]
    check(make(q, [(i * 13) % 41 for i in range(B)], 4, 2, 64, 8, seed=11, max_pages=6))


@pytest.mark.parametrize("spread", [30.0, 1e-3])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [2, 140])
def test_peaked_and_flat_scores(n, fp8, spread):
    """Scores spread over hundreds (softmax close to a maximum), and all alike."""
    s = make([n], [900], 4, 2, 128, 32, fp8, seed=12)
    s["q"] = (s["q"].float() * spread).to(torch.bfloat16)
    out = call(s)
    want, mags, owned = ref.attention(s["q"], 4, s["k_cache"], s["v_cache"], s["cu_q"], s["kv_len"], s["block_table"],
                                      k_scale=s["k_scale"], v_scale=s["v_scale"])
    # scores of spread x sum |q k| scale <= 30 x 64 are off by up to 128 x 2^-24 x 30 x 64 = 2^-6 at worst
    err = (out.double() - want).abs()
    extra = 2.0 ** -5 if spread > 1 else 0.0
    assert (err <= (2.0 ** -8 + 2.0 ** -9 + extra) * mags + 2.0 ** -8 * want.abs()).all()


@pytest.mark.parametrize("n", [1, 150])
def test_scales_of_q_at_the_ends_of_the_type(n):
    """An E4M3 cache with queries of about 2^110 and 2^-110, the softmax scale undoing it."""
    s = make([n], [300], 8, 2, 128, 16, True, seed=13)
    base = s["q"].clone()
    want = call(s, scale=2.0 ** -4)
    for e in (90, -90, 110, -110):
        s["q"] = base * 2.0 ** e
        assert torch.equal(call(s, scale=2.0 ** (-4 - e)), want)


@pytest.mark.parametrize("n", [1, 300])
def test_strided_rows_of_a_fused_projection(n):
    """Q as a column slice of a wider matrix, O with a padded row stride inside a sentinel."""
    s = make([n, 1], [n + 100, 50], 8, 2, 128, 16, seed=14)
    want = call(s)
    wide = torch.randn(n + 1, 12 * 128 + 8, device="cuda").to(torch.bfloat16)
    wide[:, 8:8 + 1024] = s["q"]
    s["q"] = wide[:, 8:8 + 1024]
    buf = torch.full((n + 2, 1024 + 64), SENTINEL, dtype=torch.bfloat16, device="cuda")
    call(s, out=buf[:n + 1, :1024])
    assert torch.equal(buf[:n + 1, :1024], want)
    assert (buf[n + 1:] == SENTINEL).all() and (buf[:, 1024:] == SENTINEL).all()


def test_pages_beyond_32_bit_offsets():
    """A cache of 2^31 + elements a side (pages interleaved, 2.2 GB each way): its last pages."""
    page, Hk, d = 16, 8, 128
    pages = (1 << 31) // (page * Hk * d) + 9
    k, v = (torch.empty(pages, page, Hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    small = make([1, 40], [70, 60], 16, Hk, d, page, seed=15)
    n = small["k_cache"].shape[0]
    k[-n:], v[-n:] = small["k_cache"], small["v_cache"]
    want = call(small)
    big = {**small, "k_cache": k, "v_cache": v, "block_table": torch.where(
        small["block_table"] >= 0, small["block_table"] + (pages - n), small["block_table"])}
    assert torch.equal(call(big), want)


@pytest.mark.parametrize("n", [1, 160])
def test_one_page_shared_by_sequences_and_repeated(n):
    """Sequences that share a prefix's pages, and one that lists a page twice."""
    s = make([n, n], [200, 200], 8, 2, 128, 8, seed=16)
    s["block_table"][1, :3] = s["block_table"][0, :3]
    s["block_table"][0, 4] = s["block_table"][0, 3]
    check(s)


@pytest.mark.parametrize("n", [1, 200])
def test_streams_graphs_and_repeats_agree(n):
    """The same call eager, again, on a side stream, and captured and replayed over changed
    lengths: bit for bit the eager results (the order of every sum is fixed by the lengths)."""
    s = make([n, n, n], [900, 333, 512], 8, 2, 128, 16, seed=17, max_pages=64)
    want = call(s)
    assert torch.equal(call(s), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [call(s, stream=side) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    g = torch.cuda.CUDAGraph()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call(s, out=out)
    for lens in ([900, 333, 512], [300, 300, 200], [n, 900, n]):
        s["kv_len"].copy_(torch.tensor(lens, dtype=torch.int32))
        s["kv_len"].clamp_(max=333 if lens[1] == 333 else 900)
        eager = call(s)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(torch.nan_to_num(out, 1e4), torch.nan_to_num(eager, 1e4))


def test_two_streams_at_once():
    """Calls of different shapes on two streams, each with its own workspace."""
    a = make([1] * 6, [2000, 30, 500, 1, 77, 900], 8, 2, 128, 16, seed=18)
    b = make([150, 20], [600, 400], 8, 4, 64, 32, True, seed=19)
    want = [call(a), call(b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(4):
        for i, s in enumerate((a, b)):
            outs[i].append(call(s, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_lens", [[1, 2], [20, 3]])
@pytest.mark.parametrize("Hq,Hk,d", [(1024, 1024, 64), (512, 512, 128), (128, 1, 128), (160, 1, 64), (512, 2, 128),
                                     (1000, 1, 64)])
def test_many_heads(Hq, Hk, d, q_lens, fp8):
    """As many key heads as fit, groups of 128 heads (a row tile's half is one token) and larger."""
    check(make(q_lens, [q_lens[0] + 70, q_lens[1] + 9], Hq, Hk, d, 16, fp8, seed=Hk))


@pytest.mark.parametrize("fp8", [False, True])
def test_many_short_chunks(fp8):
    """More sequences of many rows than the kernel weighs at once."""
    q = [17 + i % 5 for i in range(900)]
    q[7] = q[500] = q[501] = 0
    check(make(q, [n + (i * 13) % 41 for i, n in enumerate(q)], 2, 2, 64, 8, fp8, seed=20, max_pages=8))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [2, 150])
def test_a_row_of_nan_stays_alone(n, fp8):
    """The other rows are held to the formula: rows of a tile raise their maxima together, so the
    exponents that the weights are rounded at (any between the maximum and 2^8 of it are right)
    may depend on the neighbours, the error bound does not."""
    s = make([n, n], [300, 200], 8, 2, 128, 16, fp8, seed=21)
    want, mags, owned = ref.attention(s["q"], 8, s["k_cache"], s["v_cache"], s["cu_q"], s["kv_len"], s["block_table"],
                                      k_scale=s["k_scale"], v_scale=s["v_scale"])
    s["q"][1, 128:256] = float("nan")
    s["q"][n, 5] = float("inf")
    out = call(s)
    assert torch.isnan(out[1, 128:256]).all() and torch.isnan(out[n, :128]).all()
    out[1, 128:256], out[n, :128] = want[1, 128:256].to(out.dtype), want[n, :128].to(out.dtype)
    ref.assert_attention(out, want, mags, owned)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,kv", [(3, 100), (2, 6000), (200, 300), (150, 3000)])
def test_attended_nan_is_seen(n, kv, fp8):
    """A key or a value that is NaN: every row that attends it is NaN (a value: in its column)."""
    for which, cols in (("k_cache", slice(0, 64)), ("v_cache", slice(9, 10))):
        s = make([n], [kv], 2, 1, 64, 16, fp8, seed=22)
        pos = kv - n + 1
        cache = s[which].view(torch.uint8) if fp8 else s[which]
        cache[int(s["block_table"][0, pos // 16]), pos % 16, 0, 9] = 0x7F if fp8 else float("nan")
        out = call(s).reshape(n, 2, 64)
        assert torch.isnan(out[1:, :, cols]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [2, 150])
def test_scale_of_zero_averages(n, fp8):
    check(make([n, 1], [400, 77], 8, 2, 128, 16, fp8, seed=23), scale=0.0)


@pytest.mark.parametrize("n", [2, 150])
def test_workspace_contents_do_not_matter(n):
    s = make([n, 1], [4000, 77], 8, 2, 128, 16, seed=24)
    want = call(s)
    ws = mxq.attention_paged_workspace(n + 1, 2, 8, 2, 128, "cuda")
    for fill in (0xFF, 0x00, 0x3C):
        ws.fill_(fill)
        assert torch.equal(call(s, workspace=ws), want)
    with pytest.raises(mxq.MxqError):
        call(s, workspace=ws[:-256])
    with pytest.raises(ValueError, match="workspace"):
        call(s, workspace=ws[:1].expand(ws.numel()))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [8, 24, 64, 256])
@pytest.mark.parametrize("q_lens", [[2, 1, 1], [150, 129, 40]])
def test_missing_pages_of_every_size(q_lens, page, fp8):
    """Pages that are missing at the start, inside and at the end of a sequence, in tiles that hold
    other pages and in tiles without any; the memory of a page that is there but unused is NaN."""
    s = make(q_lens, [700, 1100, 333], 8, 2, 128, page, fp8, seed=25)
    n = [-(-k // page) for k in (700, 1100, 333)]
    for b, entries in enumerate(([0, n[0] // 2], [1, n[1] - 1], [0])):
        for e in entries:
            s["block_table"][b, e] = -1 if b else s["k_cache"].shape[0] + e
    s["block_table"][1, n[1] // 3:n[1] // 2] = -1
    check(s)
    check(s, causal=False)
    check(s, window=200)


@pytest.mark.parametrize("page", [8, 64])
@pytest.mark.parametrize("n", [3, 150])
def test_garbage_behind_a_window_of_an_e4m3_cache(n, page):
    """NaN bytes at every position that no row's window reaches."""
    s = make([n, 1], [600, 300], 4, 2, 128, page, True, seed=26)
    window = 77
    clean = call(s, window=window)
    for b, rows in enumerate((n, 1)):
        L = int(s["kv_len"][b])
        for j in range(L - rows - window + 1):
            for c in (s["k_cache"], s["v_cache"]):
                c.view(torch.uint8)[int(s["block_table"][b, j // page]), j % page] = 0x7F
    out = call(s, window=window)
    assert torch.isfinite(out).all() and torch.equal(out, clean)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_long_chunk_among_idle_sequences(fp8):
    """The kernel is chosen by the mean number of rows; either is right for any lengths."""
    q = [0] * 120
    q[50], q[51], q[119] = 300, 1, 7
    check(make(q, [n + 50 for n in q], 8, 2, 128, 16, fp8, seed=27))


@pytest.mark.parametrize("n", [1, 150])
def test_graphs_with_one_workspace_in_turn(n):
    """Two captured calls of different lengths share a workspace and replay one after another."""
    sets = [make([n, n], [3000, 200], 8, 2, 128, 16, seed=28), make([n, n], [n, 5000], 8, 2, 128, 16, True, seed=29)]
    want = [call(s) for s in sets]
    ws = mxq.attention_paged_workspace(2 * n, 2, 8, 2, 128, "cuda")
    outs, graphs = [torch.zeros_like(w) for w in want], []
    torch.cuda.synchronize()
    for s, o in zip(sets, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(s, out=o, workspace=ws)
        graphs.append(g)
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
