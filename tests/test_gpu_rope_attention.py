"""Norm and rotation of queries and keys ahead of the MXFP4 attention: the rotated operands held to the formula in 64
bits, the attention to the oracle's of them."""

import numpy as np
import pytest
import torch

import oracle
import paged_ref as ref
from mxfp4_block_scaled_mxq_b200 import build, inputs, mxq
from parity import assert_status_clean

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mxq.lib()
    yield
    assert_status_clean()


@pytest.mark.parametrize("row", [False, True])
@pytest.mark.parametrize("T", [1, 300])
def test_norm_rope_then_attention(T, row):
    """A video layer: one norm per head or per row, neighbouring pairs rotated, every key visible.  5e-3 of the largest
    value is the MXFP4 attention's bound (BF16 output, FP32 sums)."""
    H, d = 2, 128
    q, k = (inputs.heavy_tailed_bf16(T, H * d, seed=s, device="cuda") for s in (60, 61))
    v = inputs.normal_bf16(T, H * d, 1.0, seed=62)
    g = torch.Generator(device="cuda").manual_seed(63)
    w = (1 + 0.3 * torch.randn(H * d if row else d, generator=g, device="cuda")).to(torch.bfloat16)
    table, pos = mxq.rope_table(T, d), torch.arange(T, device="cuda")
    qo, ko = mxq.qk_norm_rope(q, k, H, H, w, w, span=mxq.MXQ_NORM_ROW if row else mxq.MXQ_NORM_HEAD, table=table,
                              style=mxq.MXQ_ROPE_PAIRS)
    got = mxq.attention_mxfp4(qo, ko, v.cuda(), H).float().cpu().numpy().reshape(T, H, d)
    for x, raw in ((qo, q), (ko, k)):
        ref.assert_rounded(x, *ref.norm_rope(raw, H, w, table, pos, 1e-6, row, True))
    want, _ = oracle.attention_mxfp4(qo.cpu(), ko.cpu(), v, H, d, np.arange(T))
    assert np.abs(got - want).max() <= 5e-3 * np.abs(want).max()
