"""A block's scale and factor, fl(MAX / amax) and fl(1 / scale), against the correctly rounded divisions for every maximum of
a binade.  The kernels that quantise activations work them out by a refined reciprocal, whose last bit hangs on the hardware's
first estimate for a handful of mantissas only: a random sample would miss them."""
import numpy as np
import pytest
import torch

from helpers import gpu

pytestmark = pytest.mark.gpu

#: binades of maxima: ordinary ones, the last one below the smallest maximum that counts (2^-100), the first above it, the
#: largest, and those whose scales lie around 1.
FIRST = {"1 to 2": 0x3f800000, "below 2^-100": 0x0d000000, "from 2^-100": 0x0d800000, "from 2^127": 0x7f000000, "from 2^8": 0x43800000,
         "from 2^15": 0x47000000}


@pytest.mark.parametrize("fmt,most,top", [(0, 448.0, 0x7e), (1, 57344.0, 0x7b)])
@pytest.mark.parametrize("binade", FIRST)
def test_every_maximum_of_a_binade(binade, fmt, most, top):
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    N, C = 1 << 20, 16
    pos = torch.arange(N, dtype=torch.int32, device=dev)[:, None].contiguous()
    q, s = torch.empty((N, C), dtype=torch.uint8, device=dev), torch.empty((1, N), device=dev)
    x = torch.zeros((N, C), device=dev)
    for first in range(FIRST[binade], FIRST[binade] + (1 << 23), N):
        amax = np.arange(first, first + N, dtype=np.uint32).view(np.float32)
        x[:, 5] = torch.from_numpy(amax).to(dev)
        fd.fp8_block_dispatch(x, fmt, pos, q, s)
        scale = np.float32(most) / np.maximum(amax, np.float32(2.0 ** -100))
        assert np.array_equal(s[0].cpu().numpy(), np.float32(1) / scale)
        if binade != "below 2^-100":
            assert torch.all(q[:, 5] == top)
        assert int((q != 0).sum()) == int((q[:, 5] != 0).sum())
