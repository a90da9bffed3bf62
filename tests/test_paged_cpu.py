"""Refusals of the norm / rotation, the cache append and the paged attention: every bad argument
is turned down on the host before anything is launched.  No kernel runs here."""

import ctypes

import pytest
import torch

from mxfp4_block_scaled_mxq_b200 import build, mxq

INV, SHAPE, ALIGN, UNSUP, CUDA = 1, 2, 3, 4, 5
FAKE = 1 << 20  # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return mxq.lib()


def cfg(**kw):
    base = dict(q_weight=FAKE, k_weight=FAKE, table=FAKE, table_rows=100, rot=128, eps=1e-6, span=0, style=0)
    return mxq.NormRope(**{**base, **kw})


def kv(**kw):
    base = dict(k=FAKE, v=FAKE, num_pages=10, page_size=16, heads=2, d=128, stride_page=16 * 256, stride_token=256,
                stride_head=128, fmt=0, k_scale=1.0, v_scale=1.0)
    return mxq.PagedKVArgs(**{**base, **kw})


def batch(**kw):
    base = dict(cu_q=FAKE, kv_len=FAKE, block_table=FAKE, batch=3, max_pages=7)
    return mxq.PagedBatchArgs(**{**base, **kw})


def ref(x):
    return None if x is None else ctypes.byref(x)


def norm_rope(L, c=None, **kw):
    a = dict(T=5, d=128, q=FAKE, Hq=4, ldq=512, qo=FAKE, ldqo=512, k=FAKE, Hk=2, ldk=256, ko=FAKE, ldko=256, pos=None)
    a.update(kw)
    return L.mxq_qk_norm_rope(ref(c or cfg()), *a.values(), None)


def append(L, c=None, cache=None, b=None, **kw):
    a = dict(T=5, k=FAKE, ldk=256, v=FAKE, ldv=256, q=None, Hq=0, ldq=0, qo=None, ldqo=0)
    a.update(kw)
    return L.mxq_kv_append(ref(c or cfg()), ref(cache or kv()), ref(b or batch()), *a.values(), None)


def attend(L, cache=None, b=None, **kw):
    a = dict(q=FAKE, T=5, Hq=8, ldq=1024)
    t = dict(causal=1, window=0, scale=0.1, ws=FAKE, wsb=1 << 40, out=FAKE, ldo=1024)
    a.update({k: v for k, v in kw.items() if k in a})
    t.update({k: v for k, v in kw.items() if k in t})
    return L.mxq_attention_paged(*a.values(), ref(cache or kv()), ref(b or batch()), *t.values(), None)


def test_valid_calls_pass_the_checks(L):
    """Without a B200 they then fail for the device; nothing is launched."""
    if torch.cuda.is_available():
        pytest.skip("the fake pointers are for hosts without a GPU")
    for st in (norm_rope(L), append(L), attend(L), append(L, q=FAKE, Hq=4, ldq=512, qo=FAKE, ldqo=512)):
        assert st in (UNSUP, CUDA)


@pytest.mark.parametrize("want,c,kw", [
    (INV, {}, dict(q=None, k=None)), (INV, {}, dict(qo=None)), (INV, {}, dict(ko=None)),
    (SHAPE, {}, dict(T=0)), (SHAPE, {}, dict(T=1 << 31)), (SHAPE, {}, dict(d=120)), (SHAPE, {}, dict(d=272)),
    (SHAPE, {}, dict(Hq=0)), (SHAPE, {}, dict(Hq=513, ldq=1 << 20, ldqo=1 << 20)),
    (ALIGN, {}, dict(ldq=504)), (ALIGN, {}, dict(ldq=516)), (ALIGN, {}, dict(q=FAKE + 8)), (ALIGN, {}, dict(ko=FAKE + 2)),
    (ALIGN, {}, dict(pos=FAKE + 2)), (ALIGN, {}, dict(ldko=128)),
    (INV, dict(span=2), {}), (INV, dict(style=-1), {}), (INV, dict(eps=-1.0), {}), (INV, dict(eps=float("nan")), {}),
    (INV, dict(table=None), {}), (INV, dict(rot=0), {}), (SHAPE, dict(rot=24), {}), (SHAPE, dict(rot=144), {}),
    (SHAPE, dict(table_rows=0), {}), (ALIGN, dict(q_weight=FAKE + 8), {}), (ALIGN, dict(table=FAKE + 4), {})])
def test_norm_rope_refusals(L, want, c, kw):
    assert norm_rope(L, cfg(**c), **kw) == want


def test_norm_rope_needs_a_configuration(L):
    assert L.mxq_qk_norm_rope(None, 5, 128, FAKE, 4, 512, FAKE, 512, None, 0, 0, None, 0, None, None) == INV


CACHE_REFUSALS = [
    (INV, dict(k=None)), (INV, dict(v=None)), (INV, dict(fmt=2)), (INV, dict(k_scale=2.0)),
    (INV, dict(fmt=1, k_scale=0.0)), (INV, dict(fmt=1, v_scale=float("inf"))), (INV, dict(fmt=1, v_scale=1e-45)),
    (SHAPE, dict(num_pages=0)), (SHAPE, dict(num_pages=(1 << 30) + 1)), (SHAPE, dict(page_size=0)),
    (SHAPE, dict(page_size=12)), (SHAPE, dict(heads=0)), (SHAPE, dict(heads=1024)), (SHAPE, dict(d=24)),
    (ALIGN, dict(stride_token=120)), (ALIGN, dict(stride_head=132)), (ALIGN, dict(stride_page=0)),
    (ALIGN, dict(fmt=1, stride_token=264)), (ALIGN, dict(stride_page=1 << 39)), (ALIGN, dict(k=FAKE + 8))]
BATCH_REFUSALS = [
    (INV, dict(cu_q=None)), (INV, dict(kv_len=None)), (INV, dict(block_table=None)), (SHAPE, dict(batch=0)),
    (SHAPE, dict(batch=(1 << 20) + 1)), (SHAPE, dict(max_pages=0)), (SHAPE, dict(max_pages=(1 << 26) + 1)),
    (ALIGN, dict(cu_q=FAKE + 2))]


@pytest.mark.parametrize("want,c", CACHE_REFUSALS)
def test_cache_refusals(L, want, c):
    assert append(L, cache=kv(**c)) == want
    assert attend(L, cache=kv(**c)) == want


@pytest.mark.parametrize("want,b", BATCH_REFUSALS)
def test_batch_refusals(L, want, b):
    assert append(L, b=batch(**b)) == want
    assert attend(L, b=batch(**b)) == want


@pytest.mark.parametrize("want,kw", [
    (INV, dict(k=None)), (INV, dict(v=None)), (INV, dict(q=FAKE, Hq=4, ldq=512)), (SHAPE, dict(T=0)),
    (ALIGN, dict(ldk=248)), (ALIGN, dict(v=FAKE + 4)), (SHAPE, dict(q=FAKE, Hq=0, ldq=512, qo=FAKE, ldqo=512)),
    (ALIGN, dict(q=FAKE, Hq=4, ldq=512, qo=FAKE, ldqo=500))])
def test_append_refusals(L, want, kw):
    assert append(L, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (INV, dict(q=None)), (INV, dict(out=None)), (INV, dict(ws=None)), (INV, dict(wsb=100)), (ALIGN, dict(ws=FAKE + 128)),
    (INV, dict(scale=float("nan"))), (INV, dict(scale=3e38)), (INV, dict(window=-1)), (INV, dict(window=5, causal=0)),
    (SHAPE, dict(window=(1 << 30) + 1)), (SHAPE, dict(Hq=7, ldq=896, ldo=896)), (SHAPE, dict(Hq=0)), (SHAPE, dict(T=0)),
    (SHAPE, dict(T=1 << 28)), (ALIGN, dict(ldo=1000)), (ALIGN, dict(ldq=1028)), (ALIGN, dict(out=FAKE + 8))])
def test_attention_refusals(L, want, kw):
    assert attend(L, **kw) == want


def test_attention_head_dimension(L):
    c = kv(d=80, stride_head=80, stride_token=160, stride_page=16 * 160)
    assert attend(L, cache=c, Hq=8, ldq=640, ldo=640) == UNSUP
    assert mxq.mxq_attention_paged_workspace_bytes(1, 1, 8, 2, 80) == -1
    assert mxq.mxq_attention_paged_workspace_bytes(1, 1, 8, 3, 128) == -1
    assert mxq.mxq_attention_paged_workspace_bytes(0, 1, 8, 2, 128) == -1
    assert mxq.mxq_attention_paged_workspace_bytes(1, 1, 8, 2, 128) > 0


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mxq.qk_norm_rope(x, x, 2, 2)
    c = torch.zeros(3, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mxq.PagedKV(c, c)
    with pytest.raises(ValueError, match="alike"):
        mxq.PagedKV(c, c[:2])
    with pytest.raises(ValueError, match="bfloat16"):
        mxq.PagedKV(c.float(), c.float())
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="cu_q"):
        mxq.PagedBatch(i, i[:3], i[:3].reshape(3, 1))


def test_struct_layouts_match_the_header():
    """ctypes structures and the C ones agree in size (a compiled check of include/mxq.h)."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = ('#include <stdio.h>\n#include <stddef.h>\n#include "mxq.h"\nint main(void){printf("%zu %zu %zu %zu %zu %zu",'
           "sizeof(mxq_norm_rope),sizeof(mxq_paged_kv),sizeof(mxq_paged_batch),offsetof(mxq_norm_rope,style),"
           "offsetof(mxq_paged_kv,v_scale),offsetof(mxq_paged_batch,max_pages));return 0;}")
    with tempfile.TemporaryDirectory() as t:
        with open(os.path.join(t, "a.c"), "w") as f:
            f.write(src)
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), "-o", os.path.join(t, "a"), os.path.join(t, "a.c")],
                       check=True)
        got = [int(x) for x in subprocess.run([os.path.join(t, "a")], check=True, capture_output=True).stdout.split()]
    want = [ctypes.sizeof(c) for c in (mxq.NormRope, mxq.PagedKVArgs, mxq.PagedBatchArgs)]
    want += [mxq.NormRope.style.offset, mxq.PagedKVArgs.v_scale.offset, mxq.PagedBatchArgs.max_pages.offset]
    assert got == want
