"""Paged attention captured into a CUDA graph and replayed over other lengths, pages and queries: at the captured
lengths bit for bit the eager result, at grown and shrunk ones finite and held to the formula in 64 bits."""

import pytest
import torch

import paged_ref as ref
from mxfp4_block_scaled_mxq_b200 import build, mxq
from parity import assert_status_clean
from test_gpu_paged_attention import SENTINEL, call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    mxq.lib()
    yield
    assert_status_clean()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 5, 200])
def test_replays_over_other_lengths(n, fp8):
    """Every sequence has pages and finite keys for its longest length; rows and pages may move between replays."""
    longest, captured = [4000, 900, 700], [900, 333, 512]
    s = make([n] * 3, longest, 8, 2, 128, 16, fp8, seed=40)
    s["kv_len"].copy_(torch.tensor(captured, dtype=torch.int32))
    kw = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    want = call(s)
    out = torch.full_like(want, SENTINEL)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call(s, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    q, table = s["q"].clone(), s["block_table"].clone()
    for step, lens in enumerate((longest, [n, 900, n], [0, 1, 700], [3999, 0, 0], captured)):
        s["kv_len"].copy_(torch.tensor(lens, dtype=torch.int32))
        s["q"].copy_(q.roll(step, 0))
        # rolled, the sequences' pages hold 700, 4000 and 900 keys
        s["block_table"].copy_(table.roll(1, 0) if lens == [n, 900, n] else table)
        out.fill_(SENTINEL)
        eager = call(s)
        g.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(out).all() and torch.equal(out, eager)
        ref.assert_attention(out, *ref.attention(s["q"], 8, s["k_cache"], s["v_cache"], s["cu_q"], s["kv_len"],
                                                 s["block_table"], **kw))
    s["q"].copy_(q)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
