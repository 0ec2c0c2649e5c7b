"""moe_route and moe_route_bwd against plain 64-bit routing: whole numbers exactly, the rest within what fp32
arithmetic may be off by."""
import numpy as np
import pytest
import torch

import moe_reference as mr
import workloads as wl
from helpers import gpu

pytestmark = pytest.mark.gpu


class Buffers:
    """Everything moe_route writes, filled with what no result is; a guard row behind each."""

    def __init__(self, fd, T, E, k, dev, ws=None):
        i32 = dict(dtype=torch.int32, device=dev)
        self.expert, self.position = torch.full((T, k), -7, **i32), torch.full((T, k), -7, **i32)
        self.weight = torch.full((T, k), -7.0, device=dev)
        self.token, self.offsets, self.counts = torch.full((T * k,), -7, **i32), torch.full((E + 1,), -7, **i32), torch.full((E,), -7, **i32)
        self.slope, self.loss = torch.full((E,), -7.0, device=dev), torch.full((1,), -7.0, device=dev)
        self.ws = torch.empty(max(16, fd.moe_route_workspace_size(T, E)), dtype=torch.uint8, device=dev) if ws is None else ws

    def run(self, fd, logits, valid=None, normalize=True, balance=True, **kw):
        fd.moe_route(logits, self.expert, self.weight, self.position, self.token, self.offsets, counts=self.counts,
                     slope=self.slope if balance else None, loss=self.loss if balance else None, workspace=self.ws, valid=valid,
                     normalize=normalize, **kw)


def host(t):
    return t.detach().double().cpu().numpy()


def check(b, l, r, balance=True):
    T, k = b.expert.shape
    for name in ("expert", "position", "offsets", "counts"):
        assert np.array_equal(getattr(b, name).cpu().numpy(), r[name]), name
    n = int(r["offsets"][-1])
    assert np.array_equal(b.token.cpu().numpy()[:n], r["token"][:n]) and np.all(b.token.cpu().numpy()[n:] == -7)
    rel = mr.route_error(l, r) if T else np.zeros(0)
    assert np.all(np.abs(host(b.weight) - r["weight"]) <= 2 * rel[:, None] * r["weight"] + 2.0 ** -120)
    if balance:
        assert np.all(np.abs(host(b.slope) - r["slope"]) <= 4 * mr.EPS * r["slope"])
        # every token's p, and T + E sequential adds of positive terms
        each = (r["slope"] * (r["p"] * rel[:, None]).sum(0)).sum() + (T + l.shape[1] + 8) * mr.EPS * abs(r["loss"])
        assert abs(float(b.loss) - r["loss"]) <= each


def logits_of(T, E, dtype, name, scale=2.0):
    l = wl.normal((T, E), scale, wl.generator(400, name), dtype)
    return l, l.double().numpy()


CASES = [(1, 1, 1), (1, 64, 6), (2, 3, 3), (5, 8, 2), (17, 9, 4), (33, 16, 16), (64, 31, 5), (65, 33, 2), (130, 64, 1), (129, 100, 8),
         (300, 256, 8), (77, 255, 32), (41, 300, 7), (40, 512, 8), (23, 1000, 32), (19, 1024, 3), (5000, 8, 2), (4865, 64, 6),
         (11001, 40, 4), (2500, 1024, 2)]


@pytest.mark.parametrize("T,E,k", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_route_and_gradient(T, E, k, dtype):
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    lt, l = logits_of(T, E, dtype, "l%d,%d" % (T, E))
    valid = (torch.rand(T, generator=wl.generator(401, "v%d" % T)) > 0.2) if T % 2 else None
    normalize = (T + E) % 3 != 0
    r = mr.route(l, k, None if valid is None else valid.numpy(), normalize)
    b = Buffers(fd, T, E, k, dev)
    ld = lt.to(dev)
    b.run(fd, ld, valid=None if valid is None else valid.to(dev), normalize=normalize)
    check(b, l, r)
    dw = wl.normal((T, k), 1.0, wl.generator(402, "g"), torch.float32)
    dloss = torch.full((1,), 3.0, device=dev)
    for dwt, dlt in ((dw, dloss), (dw, None), (None, dloss)):
        d = torch.full((T, E), 9.0, dtype=dtype, device=dev)
        fd.moe_route_bwd(ld, b.expert, b.weight, d, dweight=None if dwt is None else dwt.to(dev), slope=b.slope, dloss=dlt,
                         normalize=normalize)
        want, size = mr.route_grad(r, None if dwt is None else dwt.double().numpy(), 0.0 if dlt is None else 3.0, normalize)
        # p, both sums and the chosen experts' terms each carry the token's relative error of the magnitudes
        bound = 4 * mr.route_error(l, r)[:, None] * size + torch.finfo(dtype).eps / 2 * np.abs(want) * 1.01 + 2.0 ** -110
        assert np.all(np.abs(host(d) - want) <= bound)
        assert np.all(host(d)[~r["has"][:, 0]] == 0)


def test_ties_go_to_the_lowest_expert_and_rows_keep_the_tokens_order():
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    T, E, k = 700, 72, 5
    l = torch.randint(-2, 3, (T, E), generator=wl.generator(403, "ties")).float()
    l[::3] = 0.0            # all equal
    l[1::3][l[1::3] == 0] = -0.0  # equal to 0 all the same
    for dtype in (torch.bfloat16, torch.float32):
        b = Buffers(fd, T, E, k, dev)
        b.run(fd, l.to(dtype).to(dev))
        check(b, l.double().numpy(), mr.route(l.double().numpy(), k))


def test_closed_experts_empty_rows_and_lowest_values():
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    T, E, k = 90, 20, 4
    l = wl.normal((T, E), 1.0, wl.generator(404, "closed"), torch.float32)
    l[:, 3:19] = -torch.inf                                  # four experts left
    l[10, :] = -torch.inf                                    # none
    l[11, 1:] = -torch.inf                                   # one
    l[12, :] = torch.finfo(torch.float32).min                # a mask of the type's lowest value: all equal
    l[13, 1:] = torch.finfo(torch.float32).min
    b = Buffers(fd, T, E, k, dev)
    b.run(fd, l.to(dev))
    r = mr.route(l.double().numpy(), k)
    assert r["expert"][10].tolist() == [-1] * 4 and r["expert"][11].tolist() == [0, -1, -1, -1]
    assert r["expert"][12].tolist() == [0, 1, 2, 3]
    check(b, l.double().numpy(), r)
    d = torch.full((T, E), 9.0, device=dev)
    fd.moe_route_bwd(l.to(dev), b.expert, b.weight, d, dweight=torch.ones((T, k), device=dev), slope=b.slope,
                     dloss=torch.ones(1, device=dev))
    assert torch.isfinite(d).all() and torch.all(d[10] == 0) and torch.all(d[:10, 3:19] == 0)
    # nothing but padding: no rows, a loss of zero
    b.run(fd, l.to(dev), valid=torch.zeros(T, dtype=torch.uint8, device=dev))
    assert torch.all(b.expert == -1) and torch.all(b.offsets == 0) and torch.all(b.weight == 0) and float(b.loss) == 0
    assert torch.all(b.slope == 0)


def test_nan_and_infinite_logits_stay_with_their_token():
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    T, E, k = 40, 12, 3
    l = wl.normal((T, E), 1.0, wl.generator(405, "nan"), torch.float32)
    l[3, 5], l[7, 2], l[9, :] = torch.nan, torch.inf, torch.nan
    l[11, 4] = torch.nan                                     # padding: not looked at
    valid = torch.ones(T, dtype=torch.bool)
    valid[11] = False
    b = Buffers(fd, T, E, k, dev)
    b.run(fd, l.to(dev), valid=valid.to(dev))
    clean = l.clone()
    clean[3, 5] = clean[9, :] = -torch.inf
    want = mr.route(clean.double().numpy(), k, valid.numpy())
    assert np.array_equal(b.expert.cpu().numpy(), want["expert"])  # NaN is never chosen, infinity first
    assert want["expert"][7, 0] == 2 and np.array_equal(b.position.cpu().numpy(), want["position"])
    bad = torch.zeros(T, dtype=torch.bool)
    bad[[3, 7]] = True
    assert torch.isnan(b.weight.cpu()[bad]).all() and torch.isfinite(b.weight.cpu()[~bad]).all()
    assert torch.isnan(b.loss).all()
    d = torch.zeros((T, E), device=dev)
    fd.moe_route_bwd(l.to(dev), b.expert, b.weight, d, dweight=torch.ones((T, k), device=dev))
    assert torch.isnan(d.cpu()[bad]).all() and torch.isfinite(d.cpu()[~bad]).all() and torch.all(d[11] == 0)


def test_no_tokens_no_balance_and_repeats():
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    b = Buffers(fd, 0, 9, 2, dev)
    b.run(fd, torch.zeros((0, 9), device=dev))
    assert torch.all(b.offsets == 0) and torch.all(b.counts == 0) and torch.all(b.slope == 0) and float(b.loss) == 0
    fd.moe_route_bwd(torch.zeros((0, 9), device=dev), b.expert, b.weight, torch.zeros((0, 9), device=dev))
    T, E, k = 9000, 48, 3
    lt, l = logits_of(T, E, torch.bfloat16, "repeat")
    b = Buffers(fd, T, E, k, dev)
    b.run(fd, lt.to(dev), balance=False)
    check(b, l, mr.route(l, k), balance=False)
    assert torch.all(b.slope == -7) and torch.all(b.loss == -7)
    first = None
    for _ in range(5):  # the same bits every time
        b.run(fd, lt.to(dev))
        now = [getattr(b, n).clone() for n in ("expert", "weight", "position", "token", "slope", "loss")]
        assert first is None or all(torch.equal(x, y) for x, y in zip(first, now))
        first = now


def test_gradient_by_differences():
    """The kernels' gradient against central differences of the kernels' own forward, in fp32: the loss's third
    derivative bounds h^2, its rounding bounds 1 / h."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    T, E, k = 6, 10, 3
    lt, l = logits_of(T, E, torch.float32, "diff", 1.0)
    G = wl.normal((T, k), 1.0, wl.generator(406, "g"), torch.float32)
    for normalize in (False, True):
        b = Buffers(fd, T, E, k, dev)
        b.run(fd, lt.to(dev), normalize=normalize)
        d = torch.zeros((T, E), device=dev)
        fd.moe_route_bwd(lt.to(dev), b.expert, b.weight, d, dweight=G.to(dev), slope=b.slope, dloss=torch.full((1,), 2.0, device=dev),
                         normalize=normalize)
        order, h = b.expert.clone(), 2.0 ** -7

        def value(x):
            b.run(fd, x.to(dev), normalize=normalize)
            assert torch.equal(b.expert, order)
            return float((b.weight.double().cpu() * G).sum() + 2 * b.loss.double().cpu())

        for i in np.ndindex(T, E):
            v = torch.zeros((T, E))
            v[i] = h
            # |f'''| <= 8 (sum of |G| of the token + 2 slopes); a value's rounding: 300 units of the sum of magnitudes
            size = float(G[i[0]].abs().sum()) + 2 * E
            tol = h * h / 6 * 8 * size + 300 * mr.EPS * (float(G.abs().sum()) + 4 * E) / h
            try:
                diff = (value(lt + v) - value(lt - v)) / (2 * h)
            except AssertionError:
                continue  # a tie within h: the choice changes
            assert abs(diff - float(d[i])) <= tol
