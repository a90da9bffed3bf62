"""The tensors of a batch and of its cache lie on one device: what the binding checks of it on the host, with
stand-ins that only report a device.  No kernel runs here."""

import pytest
import torch

from mxfp4_block_scaled_mxq_b200 import mxq


class OnDevice:
    """What the checks look at, of a contiguous CUDA tensor on device `index`."""

    is_cuda = True

    def __init__(self, index, *shape, dtype=torch.int32):
        self.device, self.shape, self.dtype = torch.device("cuda", index), torch.Size(shape), dtype

    def get_device(self):
        return self.device.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


@pytest.fixture(autouse=True, params=[0, 1])
def current(request, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: request.param)
    return request.param


@pytest.mark.parametrize("devices", [(0, 0, 1), (0, 1, 0), (1, 0, 0), (1, 1, 0), (1, 0, 1), (0, 1, 1)])
def test_batch_of_two_devices_is_refused(devices):
    """Whichever of the two is the current one."""
    a, b, c = devices
    with pytest.raises(ValueError, match="cuda:"):
        mxq.PagedBatch(OnDevice(a, 4), OnDevice(b, 3), OnDevice(c, 3, 7))


@pytest.mark.parametrize("device", [0, 1])
def test_batch_of_one_device_is_made_from_any_current_device(device):
    b = mxq.PagedBatch(OnDevice(device, 4), OnDevice(device, 3), OnDevice(device, 3, 7))
    assert (b.args.batch, b.args.max_pages) == (3, 7)


def test_operands_of_another_device_are_refused(current):
    """Norm weights and rotation tables, whose device is compared with the call's."""
    here, there = current, 1 - current
    mxq._weight(OnDevice(here, 128, dtype=torch.bfloat16), 128, here, "k_weight")
    with pytest.raises(ValueError, match="k_weight"):
        mxq._weight(OnDevice(there, 128, dtype=torch.bfloat16), 128, here, "k_weight")
    with pytest.raises(ValueError, match="table"):
        mxq._norm_rope(1, 1, 128, None, None, 1e-6, 0, OnDevice(there, 9, 128, dtype=torch.float32), 0, here)


def test_batch_on_the_host_is_refused():
    i = torch.zeros(4, dtype=torch.int32)
    for cu, lens, table in ((OnDevice(0, 4), OnDevice(0, 3), i[:3].reshape(3, 1)),
                            (OnDevice(0, 4), i[:3], OnDevice(0, 3, 1)), (i, OnDevice(0, 3), OnDevice(0, 3, 1))):
        with pytest.raises(ValueError, match="CUDA"):
            mxq.PagedBatch(cu, lens, table)
