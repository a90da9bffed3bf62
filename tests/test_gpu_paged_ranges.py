"""Paged attention (mxq_attention_paged) at the ends of its numbers' ranges, against the formula in 64 bits: one key
over a flat tail of far smaller weights, in the few-row and the many-row kernel."""

import math

import pytest
import torch

import paged_ref as ref
from mxfp4_block_scaled_mxq_b200 import build, mxq
from parity import assert_status_clean
from test_gpu_paged_attention import call

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
