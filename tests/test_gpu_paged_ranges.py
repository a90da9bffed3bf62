"""Paged attention (mxq_attention_paged) at the ends of its numbers' ranges, against the formula in 64 bits: one key
over a flat tail of far smaller weights, and queries with an outlier channel, in the few-row and the
many-row kernel."""

import math

import pytest
import torch

import paged_ref as ref
from mxfp4_block_scaled_mxq_b200 import build, mxq
from parity import assert_status_clean
from test_gpu_paged_attention import call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mxq.lib()
    yield
    assert_status_clean()


@pytest.mark.parametrize("at", [0, 1])
@pytest.mark.parametrize("L", [100, 1000])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [8, 14, 40])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_strong_key_over_a_flat_tail(fp8, n, d, L, at):
    """One key of weight 1 (first or last) with a value of 0, all others of weight 2^-t and value 1: the result
    is the tail's share alone, so weights that vanish from the product but not from the sum are seen at once.

    A weight e (relative to the largest, which is 1) is rounded by 2^-8 e at most (BF16), or by 2^-11 e
    and 2^-32 absolute (FP16 below its normal range, times 2^7); the result to BF16.  Scores are exact but
    for the softmax scale, and t <= 33 in FP32 is off by under 2^-18, the exponential, sums and division
    by some more 2^-18: 2^-14 of the result in all."""
    g = torch.Generator(device="cuda").manual_seed(n)
    page, pages = 16, -(-L // 16)
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    k, v = torch.zeros(2, pages, page, 1, d, device="cuda").unbind(0)
    v = v + 1.0
    i = 0 if at == 0 else L - 1
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    k[table[0, i // page], i % page, 0, 5] = 1.0
    v[table[0, i // page], i % page] = 0.0
    q = torch.zeros(n, d, device="cuda")
    q[:, 5] = 15.0 + 0.25 * torch.randint(0, 73, (n,), generator=g, device="cuda")  # t, exact in BF16
    s = dict(q=q.to(torch.bfloat16), Hq=1, k_cache=k.to(dtype), v_cache=v.to(dtype), k_scale=1.0, v_scale=1.0,
             cu_q=torch.tensor([0, n], dtype=torch.int32, device="cuda"),
             kv_len=torch.tensor([L], dtype=torch.int32, device="cuda"), block_table=table)
    out = call(s, scale=math.log(2.0), causal=False)
    want, mags, _ = ref.attention(s["q"], 1, s["k_cache"], s["v_cache"], s["cu_q"], s["kv_len"], table, causal=False,
                                  scale=math.log(2.0))
    weights = 2.0 ** -11 * mags + 2.0 ** -32 * L if fp8 else 2.0 ** -8 * mags
    err = (out.double() - want).abs()
    tol = weights + (2.0 ** -8 + 2.0 ** -14) * want
    assert (err <= tol).all(), (float((err / tol).max()), float((err / want).max()))


def _outlier_channel(n, d, low, ratio, seed):
    """An E4M3 cache and queries whose channel 7 is `ratio` times the others, with keys small in it.  `low`: the
    least magnitude of the other channels, whose largest is below 4 (0: a normal's values)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    L, page = 300, 16
    pages = -(-L // page)
    k, v = torch.randn(2, pages, page, 2, d, generator=g, device="cuda").unbind(0)
    k[..., 7] /= ratio
    k, v = ((c / 0.02).clamp(-448, 448).to(torch.float8_e4m3fn) for c in (k, v))
    q = torch.randn(n, 2 * d, generator=g, device="cuda")
    if low:
        q = q.sign() * (low + q.abs()).clamp(max=4 - 2.0 ** -6)
    for h in range(2):
        q[:, h * d + 7] = ratio * (1 + 0.9 * torch.rand(n, generator=g, device="cuda"))
    return dict(q=q.to(torch.bfloat16), Hq=2, k_cache=k, v_cache=v, k_scale=0.02, v_scale=0.02,
                cu_q=torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                kv_len=torch.tensor([L], dtype=torch.int32, device="cuda"),
                block_table=torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None])


def _against_formula(s, query_error):
    """query_error(row's largest): how far a query value may be off.  A score is then off by that x scale x sum |K_j|
    over the channels, at most D over the keys; a weight and the sum of the weights change by e^D each."""
    out = call(s)
    want, mags, _ = ref.attention(s["q"], 2, s["k_cache"], s["v_cache"], s["cu_q"], s["kv_len"], s["block_table"],
                                  k_scale=0.02, v_scale=0.02)
    d = s["q"].shape[1] // 2
    big = s["q"].double().reshape(-1, 2, d).abs().amax(2)
    keys = (s["k_cache"].float().double() * 0.02).abs().sum(3).amax((0, 1))
    far = torch.expm1(2 * query_error(big) * keys * d ** -0.5).repeat_interleave(d, 1)
    # the weights' and the result's rounding and FP32 scores as in ref.assert_attention
    tol = (2.0 ** -8 + 2.0 ** -9 + far) * mags + 2.0 ** -8 * want.abs()
    err = (out.double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,bits,off", [(3, 17, 25), (14, 17, 25), (40, 9, 17), (300, 9, 17)])
def test_queries_with_an_outlier_channel(n, bits, off, d):
    """An E4M3 cache: queries are exact down to 2^-bits of their row's largest value (few rows 2^-17, many 2^-9) and
    off by 2^-off of it at most below."""
    exact = 2.0 ** (bits - 1)  # 1 / 1.9 of it is above 2^-bits
    _against_formula(_outlier_channel(n, d, 1.0, exact, n), lambda big: 0.0 * big)
    for ratio in (2.0 ** 9, 2.0 ** 11):
        _against_formula(_outlier_channel(n, d, 0.0, ratio, n + 1), lambda big: 2.0 ** -off * big)


def _time(f, reps):
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * reps)]
    for a, b in zip(events[::2], events[1::2]):
        a.record()
        f()
        b.record()
    torch.cuda.synchronize()
    return sorted(a.elapsed_time(b) for a, b in zip(events[::2], events[1::2]))[reps // 2]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [20, 130])
def test_rows_that_are_not_there_cost_no_time(n, fp8):
    """Rows behind the last sequence that hold NaN, in the same tile as rows that are there: they change neither the
    result nor, by more than a twentieth, the time."""
    pad, Hk = 256 - n, 8
    s = make([n], [60000], Hk, Hk, 128, 16, fp8, pad=pad, seed=30)
    other = {**s, "q": s["q"].clone()}
    s["q"][n:], other["q"][n:] = 0.0, float("nan")
    ws = mxq.attention_paged_workspace(n + pad, 1, Hk, Hk, 128, "cuda")
    outs = [torch.zeros_like(s["q"]) for _ in range(2)]
    ratios = []
    for _ in range(5):  # clocks move: the least of some pairs taken in turn
        zero, nan = (_time(lambda: call(x, out=o, workspace=ws), 30) for x, o in zip((s, other), outs))
        ratios.append(nan / zero)
    assert torch.equal(outs[0][:n], outs[1][:n])
    assert min(ratios) < 1.05, ratios


@pytest.mark.parametrize("kv", [60, 900])
@pytest.mark.parametrize("n", [3, 14, 150])
def test_an_infinite_key(n, kv):
    """A BF16 key with an infinity in one channel: rows whose query is positive there are NaN, rows whose query
    is negative do not attend it, whichever tile or part it is in."""
    for pos in (0, kv // 2, kv - 1):
        s = make([n], [kv], 2, 2, 64, 16, seed=31)
        s["k_cache"][int(s["block_table"][0, pos // 16]), pos % 16, 0, 9] = float("inf")
        out = call(s, causal=False)
        want, mags, _ = ref.attention(s["q"], 2, s["k_cache"], s["v_cache"], s["cu_q"], s["kv_len"], s["block_table"],
                                      causal=False)
        up = s["q"][:, 9] > 0
        assert torch.isnan(out[up, :64]).all() and up.any() and not up.all()
        out[up, :64], want[up, :64], mags[up, :64] = 0.0, 0.0, 1.0
        ref.assert_attention(out, want, mags, torch.ones(n, dtype=torch.bool, device="cuda"))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 14, 20])
@pytest.mark.parametrize("fp8", [False, True])
def test_sums_over_millions_of_keys(fp8, n, d):
    """As many sequences as workers, so that each one's 4 x 2^20 keys (one page, four times) are added up in one place:
    positive values, whose sums only grow.  Four copies of the keys have the result of one."""
    g = torch.Generator(device="cuda").manual_seed(n + d)
    page, times = 1 << 20, 4
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    k = torch.randn(1, page, 1, d, generator=g, device="cuda").to(dtype)
    v = (1 + torch.rand(1, page, 1, d, generator=g, device="cuda")).to(dtype)
    B = torch.cuda.get_device_properties(0).multi_processor_count * (8 if n <= 16 else 1)
    q = torch.randn(n, d, generator=g, device="cuda").to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = mxq.PagedBatch(torch.arange(B + 1, **i32) * n, torch.full((B,), times * page, **i32),
                           torch.zeros(B, times, **i32))
    out = mxq.attention_paged(q.repeat(B, 1), 1, mxq.PagedKV(k, v), batch, causal=False)
    want, mags, owned = ref.attention(q, 1, k, v, torch.tensor([0, n], **i32), torch.tensor([page], **i32),
                                      torch.zeros(1, 1, **i32), causal=False)
    ref.assert_attention(out, *(x.repeat(B, 1) for x in (want, mags)), owned.repeat(B))


@pytest.mark.parametrize("n", [1, 14, 20, 150])
@pytest.mark.parametrize("fp8", [False, True])
def test_one_sequence_of_many_millions_of_keys(fp8, n):
    """A unit in parts by all workers, each long enough to be added up in several runs, with a length that ends
    inside a page (one page of 2^20 tokens, listed 80 times): key j of the page counts 80 or 79 times."""
    g = torch.Generator(device="cuda").manual_seed(n)
    page, times, d = 1 << 20, 80, 64
    L = times * page - 12345
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    k, v = (torch.randn(1, page, 1, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn(n, d, generator=g, device="cuda").to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = mxq.PagedBatch(torch.tensor([0, n], **i32), torch.tensor([L], **i32), torch.zeros(1, times, **i32))
    out = mxq.attention_paged(q, 1, mxq.PagedKV(k, v), batch, causal=False)
    keys, vals = k[0, :, 0].float().double(), v[0, :, 0].float().double()
    counts = torch.where(torch.arange(page, device="cuda") < page - 12345, times, times - 1).double()
    want, mags = torch.empty(2, n, d, dtype=torch.float64, device="cuda").unbind(0)
    for i in range(0, n, 32):
        w = torch.softmax(q[i:i + 32].double() @ keys.T * d ** -0.5 + counts.log(), 1)
        want[i:i + 32], mags[i:i + 32] = w @ vals, w @ vals.abs()
    ref.assert_attention(out, want, mags, torch.ones(n, dtype=torch.bool, device="cuda"))
