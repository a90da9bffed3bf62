"""Workers of the few-row paged attention: every key head that a call may have needs one.  The kernels' own
constants and host arithmetic, compiled and run without a GPU."""

import os
import subprocess

import pytest

from mxfp4_block_scaled_mxq_b200 import build

SOURCE = """
#include <cstdio>
#include "paged_decode.cuh"
int main() {
  for (int sms = 1; sms <= 160; ++sms)
    for (int heads = 1; heads <= 1024; ++heads)
      std::printf("%d %d %d %d\\n", sms, heads, mxq::dec_workers(sms), mxq::dec_covers(sms, heads));
}
"""


@pytest.fixture(scope="module")
def cover(tmp_path_factory):
    """{(SMs, key heads): (workers, accepted)}"""
    t = tmp_path_factory.mktemp("workers")
    (t / "a.cu").write_text(SOURCE)
    subprocess.run([build.nvcc(), "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-I", build.CSRC, "-I",
                    os.path.join(build.ROOT, "include"), "-o", str(t / "a"), str(t / "a.cu")], check=True)
    lines = subprocess.run([str(t / "a")], check=True, capture_output=True, text=True).stdout.split("\n")
    return {(s, h): (w, bool(c)) for s, h, w, c in (map(int, x.split()) for x in lines if x)}


def test_accepted_calls_have_a_share_of_every_head(cover):
    """The kernel divides each head's line into up to workers / heads shares: none is an empty output."""
    for (_, heads), (workers, accepted) in cover.items():
        assert accepted == (workers // heads >= 1)


def test_a_whole_device_takes_every_head_count(cover):
    assert all(accepted for (sms, _), (_, accepted) in cover.items() if sms >= 128)
    assert not cover[127, 1024][1] and not cover[74, 600][1] and cover[74, 592][1]
