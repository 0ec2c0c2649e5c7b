"""The expert layer's gradients term by term: each expert, each half of the gated weights, and the logits' two sources on their
own, so that a term which is missing or wrongly scaled shows; and routing's gradient against differences, every element."""
import numpy as np
import pytest
import torch

import moe_reference as mr
import workloads as wl
from helpers import gpu
from test_gpu_blockmoe import _whole, inputs, make
from test_gpu_route import Buffers

pytestmark = pytest.mark.gpu

#: Root mean square of e4m3's rounding, relative: uniform within half a step, which is 2^-4 of a value at most.
RMS = 2.0 ** -4 / 3 ** 0.5


def noise(n):
    """What n quantised operands make of a result's norm: errors of random sign add up as their squares.  Half as much again:
    an activation's relative slope 1 + a (1 - s) or 1 + a phi / Phi, at most 1.3 where its values are not small."""
    return 1.5 * n ** 0.5 * RMS


def apart(a, b):
    a = a.double().cpu()
    assert torch.isfinite(a).all() and b.norm() > 0
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("act", range(4))
def test_every_term_of_the_layers_gradient(act):
    dev = gpu()
    T, E, H, F, k = 400, 4, 256, 256, 2
    x, logits, w1, w2, dy = inputs(T, E, H, F, k, act >= 2, "terms")
    moe = make(w1, w2, T, k, act, dev)
    dloss = 0.25
    want, _ = _whole(x, logits, w1, w2, k, act, dy, 0.0)
    y = moe.forward(x.to(dev), logits.to(dev)).clone()
    dx, dl, dw1, dw2 = (t.clone() for t in moe.backward(dy.to(dev)))  # outputs are valid until the next call
    assert apart(y, want[0]) <= noise(4) and apart(dx, want[1]) <= noise(8) and apart(dl, want[2]) <= noise(4)
    halves = [slice(0, F), slice(F, 2 * F)] if act >= 2 else [slice(0, F)]
    for e in range(E):
        assert apart(dw2[e], want[4][e]) <= noise(8), e
        for h in halves:
            assert apart(dw1[e, h], want[3][e, h]) <= noise(8), (e, h)
    for token in range(0, T, 40):  # a token's experts weigh in with their weights
        assert apart(y[token], want[0][token]) <= 2 * noise(4) and apart(dx[token], want[1][token]) <= 2 * noise(8)
    # the balance loss alone: nothing is quantised, bf16 rounds the result
    zero = torch.zeros_like(dy)
    alone, _ = _whole(x, logits, w1, w2, k, act, zero, dloss)
    moe.forward(x.to(dev), logits.to(dev))
    _, of_loss, _, _ = moe.backward(zero.to(dev), torch.full((1,), dloss, device=dev))
    got, ref = of_loss.double().cpu(), alone[2]
    assert torch.all((got - ref).abs() <= 2.0 ** -8 * 1.01 * ref.abs() + 2.0 ** -17 * ref.abs().max())
    # and both: their sum, with the sum's own rounding and those of its two parts
    dl = dl.double().cpu()
    moe.forward(x.to(dev), logits.to(dev))
    _, both, _, _ = moe.backward(dy.to(dev), torch.full((1,), dloss, device=dev))
    both = both.double().cpu()
    assert torch.all((both - dl - got).abs() <= 2.0 ** -8 * 1.01 * (both.abs() + dl.abs() + got.abs()) + 2.0 ** -17 * dl.abs().max())


@pytest.mark.parametrize("normalize", [False, True])
def test_routing_gradient_by_differences_of_every_element(normalize):
    """Central differences of the kernels' own forward pass.  A token's logits are 0.1 apart, more than the differences' 2 h = 1/64:
    the choice never changes and every element is compared."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    T, E, k, h = 6, 10, 3, 2.0 ** -7
    g = wl.generator(440, "diff")
    lt = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).float() * 0.35 + wl.normal((T, E), 0.03, g, torch.float32).clamp(-0.1, 0.1)
    G = wl.normal((T, k), 1.0, g, torch.float32)
    gaps = lt.sort(1).values.diff(dim=1)
    assert float(gaps.min()) > 0.1
    b = Buffers(fd, T, E, k, dev)
    b.run(fd, lt.to(dev), normalize=normalize)
    d = torch.zeros((T, E), device=dev)
    fd.moe_route_bwd(lt.to(dev), b.expert, b.weight, d, dweight=G.to(dev), slope=b.slope, dloss=torch.full((1,), 2.0, device=dev),
                     normalize=normalize)
    order, weight, loss = b.expert.clone(), b.weight.cpu(), float(b.loss)

    def value(x):
        b.run(fd, x.to(dev), normalize=normalize)
        assert torch.equal(b.expert, order)
        return float((b.weight.double().cpu() * G).sum() + 2 * b.loss.double().cpu())

    compared = 0
    for i in np.ndindex(T, E):
        v = torch.zeros((T, E))
        v[i] = h
        # Only this token's weights and probabilities change.  A softmax's third derivative is 1/8 at most.  Rounding: its
        # weights and p by 90 units of 2^-24 (2 d + 80, d < 4: the difference to the maximum, 2^x, sums, a division), the sums
        # over T tokens and E experts by one each and a few for the slopes' product.
        own, slope = float((G[i[0]].abs() * weight[i[0]]).sum()), float(b.slope.max())
        tol = h * h / 6 * (float(G[i[0]].abs().sum()) + 4 * slope) / 8 + mr.EPS * (90 * own + 2 * 90 * slope + 2 * (T + E + 8) * loss) / h
        diff = (value(lt + v) - value(lt - v)) / (2 * h)
        assert abs(diff - float(d[i])) <= tol
        compared += abs(float(d[i])) > 2 * tol
    assert compared >= T * k  # and the bound says something of the elements that carry most
