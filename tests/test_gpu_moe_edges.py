"""Expert routing, token exchange and activations kept in 8 bits where their arithmetic or their indices reach an end."""
import numpy as np
import pytest
import torch

import moe_reference as mr
import workloads as wl
from helpers import gpu
from test_gpu_route import Buffers, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [257, 300, 512, 640, 1000, 1024])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_choices_far_apart_in_one_lane(E, dtype):
    """Logits of both signs and all sizes side by side: some large, the others large and negative, the type's lowest value
    or -infinity, so that the choices run through every kind of neighbour among a lane's experts."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    T, k = 300, 32
    g = wl.generator(430, "far%d" % E)
    l = wl.normal((T, E), 6.0, g, torch.float32).to(dtype)
    few = torch.rand((T, E), generator=g) < 20 / E
    low, none = torch.tensor(torch.finfo(dtype).min, dtype=dtype), torch.tensor(-torch.inf, dtype=dtype)
    l[:100] = torch.where(few[:100], l[:100].abs() + 2, -l[:100].abs() - 2)
    l[100:160] = torch.where(few[100:160], l[100:160].abs() + 2, low)
    l[160:200] = torch.where(few[160:200], l[160:200].abs() + 2, none)
    l[200:240] = torch.where(few[200:240], 1e38 * l[200:240], low)
    r = mr.route(l.double().numpy(), k)
    assert (r["expert"][:160] >= 0).all() and (r["expert"][160:200] < 0).any()
    b = Buffers(fd, T, E, k, dev)
    b.run(fd, l.to(dev))
    for name in ("expert", "position", "offsets", "counts"):
        assert np.array_equal(getattr(b, name).cpu().numpy(), r[name]), name
    n = int(r["offsets"][-1])
    assert np.array_equal(b.token.cpu().numpy()[:n], r["token"][:n])
    # 1e38 times some of the logits is infinity: those tokens' weights are NaN, as softmax's are
    w, rel = host(b.weight), mr.route_error(l.double().numpy(), r)
    assert np.array_equal(np.isnan(w), np.isnan(r["weight"]))
    fine = ~np.isnan(r["weight"][:, 0])
    assert fine[:200].all() and np.all((np.abs(w - r["weight"]) <= 2 * rel[:, None] * r["weight"] + 2.0 ** -120)[fine])
