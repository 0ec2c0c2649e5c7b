"""The activations of fp8_block_act and fp8_block_dact over the whole range of their argument, to a relative error.

A block that holds one value says by its factor what that value was in fp32: factor = fl(1 / fl(MAX / amax)), so that
factor * MAX is amax to 3 roundings (3 units of 2^-24).  The checkpoint's codes are 1 or -1 and its factors |a|, so that the
decoded argument is a itself."""
import math

import numpy as np
import pytest
import torch

import block_reference as br
from helpers import gpu

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
C = 128  # one block a matrix and row
GELU, SILU, GEGLU, SWIGLU = range(4)


def truth(a, kind):
    """act(a) and its derivative in 64 bits."""
    a = np.asarray(a, np.float64)
    if kind in (GELU, GEGLU):
        cdf = 0.5 * np.array([math.erfc(-x / math.sqrt(2)) for x in a])
        return a * cdf, cdf + a * np.exp(-a * a / 2) / math.sqrt(2 * math.pi)
    z = np.exp(-np.abs(a))
    s, c = np.where(a >= 0, 1, z) / (1 + z), np.where(a >= 0, z, 1) / (1 + z)  # the sigmoid and 1 less it
    return a * s, s + a * s * c


def forward(fd, dev, a, kind, fmt=0):
    """The codes and factors of act(a) (u = 1 where gated): a row for each argument."""
    R = a.numel()
    h = a[:, None].expand(R, C)
    if kind >= GEGLU:
        h = torch.cat([h, torch.ones((R, C))], 1)
    q, s = torch.empty((R, C), dtype=torch.uint8, device=dev), torch.empty((1, R), device=dev)
    fd.fp8_block_act(h.contiguous().to(dev), kind, fmt, q, s)
    return q.cpu(), s.cpu()[0]


def backward(fd, dev, a, kind, fmt=0, dg=1.0, offsets=None):
    """What fp8_block_dact writes for these arguments, u = 1 where gated, and dg everywhere; the column sums only without groups."""
    R, gated = a.numel(), kind >= GEGLU
    W = 2 * C if gated else C
    hq, hs = torch.full((R, W), 0x38, dtype=torch.uint8), torch.ones((W // 128, R))
    hq[a < 0, :C] = 0xb8
    hs[0] = a.abs()
    T = fd.fp8_block_padded_rows(R, 0 if offsets is None else offsets.numel() - 1)
    u8, f32 = dict(dtype=torch.uint8, device=dev), dict(device=dev)
    b = dict(dh_q=torch.empty((R, W), **u8), dh_s=torch.empty((W // 128, R), **f32), dh_qt=torch.empty((W, T), **u8),
             dh_st=torch.empty((T // 128, W), **f32), g_qt=torch.empty((C, T), **u8), g_st=torch.empty((T // 128, C), **f32))
    if offsets is None:
        b.update(dbias=torch.empty(W, **f32), workspace=torch.empty(fd.fp8_cast_workspace_size(R, W), **u8))
    fd.fp8_block_dact(torch.full((R, C), dg, device=dev), hq.to(dev), 0, hs.to(dev), kind, fmt,
                      offsets=None if offsets is None else offsets.to(dev), **b)
    return {k: v.cpu() for k, v in b.items()}


def alone(n):
    """Groups of one row each."""
    return torch.arange(n + 1, dtype=torch.int32)


@pytest.mark.parametrize("kind", range(4))
def test_large_arguments(kind):
    """act(a) = a and act'(a) = 1 for large a, act(a) = act'(a) = 0 for large -a, however large: along the rows, transposed
    and in the column sums.  8 units of 2^-24: the reading's three, a sum or a product each in Phi or the sigmoid, and its use."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    a = torch.tensor([20.0, 1e3, 2050.0, 1e4, 1e6, 2.0 ** 24 - 1, 2.0 ** 24 + 2, 3e7, 1e9, 1e20, 1e38])
    v = a.double().numpy()
    y, d = truth(v, kind)

    def near(got, want, what):
        assert np.all(np.abs(got.double().numpy() * 448 - want) <= 8 * EPS * want), (what, got * 448)

    q, s = forward(fd, dev, a, kind)
    assert torch.all(q == 0x7e)
    near(s, y, "g")
    b = backward(fd, dev, a, kind)
    near(b["dh_s"][0], d, "dh along the rows")
    assert abs(float(b["dbias"][0]) - a.numel()) <= 16 * a.numel() * EPS
    if kind >= GEGLU:
        near(b["dh_s"][1], y, "dh of u along the rows")
    b = backward(fd, dev, a, kind, offsets=alone(a.numel()))
    near(b["dh_st"][:, 0], d, "dh transposed")
    near(b["g_st"][:, 0], y, "g transposed")
    # nothing is left on the other side: blocks of zeros, whose factor is 1
    a = -a[1:]
    b = backward(fd, dev, a, kind)
    assert torch.all(b["dh_s"] == 1) and torch.all(b["dh_q"] & 0x7f == 0) and torch.all(b["dbias"] == 0)
    q, s = forward(fd, dev, a, kind)
    assert torch.all(s == 1) and torch.all(q & 0x7f == 0)


SMALLEST = 2.0 ** -149


@pytest.mark.parametrize("kind", range(4))
@pytest.mark.parametrize("fmt", [0, 1])
def test_results_too_small_for_a_factor_of_their_own(kind, fmt):
    """Rows (and groups of one row) whose results are all below 2^-100, GELU's into the subnormal numbers (SiLU's are zero
    below -87.3, where its sigmoid is subnormal): they have the factor of a maximum of 2^-100, not that of zeros, and E5M2,
    which reaches 2^-16 / 57344 of that, codes for the results.

    A result is off by what the subnormal factors in it are: a times e R, each to half a step, so (|a| + 1) halves (the
    derivative's sum, at most 5.6 e: four times that), and 1e-4 relative, far below half a code (2^-4, 2^-3).  Results below
    that may be zero."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    lo, hi = (-14.8, -12.4) if kind in (GELU, GEGLU) else (-87.0, -72.0)
    a = torch.linspace(lo, hi, 400)
    v = a.double().numpy()
    y, d = truth(v, kind)
    most, half, sub = (448.0, 2.0 ** -4, 2.0 ** -10) if fmt == 0 else (57344.0, 2.0 ** -3, 2.0 ** -17)
    f8 = torch.float8_e4m3fn if fmt == 0 else torch.float8_e5m2
    scale = np.float32(most) / np.float32(2.0 ** -100)
    factor = float(np.float32(1) / scale)

    def check(q, s, want, what, most_of=2):
        q, s = q.view(f8).double().numpy(), s.double().numpy()
        err = most_of * (np.abs(v) + 1) * SMALLEST + 1e-4 * np.abs(want)
        sure = np.abs(want) > err  # not zero in fp32
        tiny = sure & (np.abs(want) < 2.0 ** -101)
        assert tiny.sum() > 100 and np.all(s[tiny] == factor), (what, s[tiny])
        assert np.all((s == factor) | (s == 1) | ~(np.abs(want) < 2.0 ** -101)), what
        off = np.abs(q * s[:, None] - want[:, None])
        assert np.all((off <= (half * np.abs(want) + sub * factor + err)[:, None] * 1.001)[s != 1]), what
        if fmt == 1:
            seen = sure & (np.abs(want) > 2.0 ** -16 / scale)
            assert np.all(q[seen] != 0) and (kind in (SILU, SWIGLU) or (seen & (np.abs(want) < 2.0 ** -126)).sum() > 5), what

    check(*forward(fd, dev, a, kind, fmt), y, "g")
    b = backward(fd, dev, a, kind, fmt)
    check(b["dh_q"][:, :C], b["dh_s"][0], d, "dh", 4)
    if kind >= GEGLU:
        check(b["dh_q"][:, C:], b["dh_s"][1], y, "dh of u")
    b = backward(fd, dev, a, kind, fmt, offsets=alone(a.numel()))
    check(b["dh_qt"][:C, ::128].t().contiguous(), b["dh_st"][:, 0], d, "dh transposed", 4)
    if fmt == 0:  # the activation's transposed codes are of the checkpoint's format
        check(b["g_qt"][:, ::128].t().contiguous(), b["g_st"][:, 0], y, "g transposed")


@pytest.mark.parametrize("kind", [GELU, GEGLU])
def test_gelu_of_infinities_in_the_checkpoint(kind):
    """A factor of infinity in the checkpoint (codes 1 and -1): the derivative has its limits, 1 and 0; NaN stays NaN."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    b = backward(fd, dev, torch.tensor([float("inf"), float("-inf"), float("nan"), 2.0]), kind)
    v = b["dh_q"][:, :C].view(torch.float8_e4m3fn).float()
    s = b["dh_s"][0]
    assert torch.all(v[0] == 448) and torch.all(v[1] == 0) and torch.all(torch.isnan(v[2])) and torch.all(v[3] == 448)
    assert abs(float(s[0]) * 448 - 1) <= 3 * EPS and s[1] == 1 and s[2] == 1
    g = b["g_qt"][0, :4].view(torch.float8_e4m3fn).float()
    assert g[0] == 448 and torch.isnan(g[1]) and torch.isnan(g[2]) and g[3] == 448


@pytest.mark.parametrize("kind", range(4))
def test_relative_errors(kind):
    """act(a) and act'(a) against 64 bits over the range of results that have a factor of their own, in units of 2^-24 with 3 for
    the reading.  E bounds the relative error of the exponential, R that of the ratio (12).

    GELU: E = 1.25 a^2 + 9.  y: E + R + 2 (the smaller part of 1 - e R for a > 0).  The derivative's small part w = phi |a| - Phi(-|a|)
    is E + 2 of |w|, R + 1 of Phi(-|a|) and 1 of phi |a| off, the sum and the product with dg 2 of the result.
    SiLU: the exponential is 1.25 |a| + 4 off, 1 + z one unit, its reciprocal two: the sigmoid s by S = (1.25 |a| + 4) (1 - s) + 3,
    or z where 1 + z is 1.  1 - s is s S off and half a step of its own; the derivative s + a s (1 - s)."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    lo, hi = (-11.3, 11.3) if kind in (GELU, GEGLU) else (-65.0, 40.0)
    near = torch.linspace(-3, 3, 3001)
    a = torch.cat([torch.linspace(lo, hi, 3000), near[near != 0], torch.logspace(-20, -1, 200), -torch.logspace(-20, -1, 200)])
    v = a.double().numpy()
    y, d = truth(v, kind)
    m = np.abs(v)
    if kind in (GELU, GEGLU):
        tail = 0.5 * np.array([math.erfc(x / math.sqrt(2)) for x in m])
        phi = m * np.exp(-m * m / 2) / math.sqrt(2 * math.pi)
        rel = 1.25 * m * m + 23
        ey = np.abs(y) * (np.where(v < 0, rel, 2 + rel * tail / (1 - tail)) + 3)
        ed = (1.25 * m * m + 11) * np.abs(phi - tail) + 13 * tail + phi + 5 * np.abs(d)
    else:
        z = np.exp(-m)
        s, c = np.where(v >= 0, 1, z) / (1 + z), np.where(v >= 0, z, 1) / (1 + z)
        S = np.where((v > 0) & (z < 2.0 ** -25), z / EPS, (1.25 * m + 4) * c + 3)
        ey = np.abs(y) * (S + 1 + 3)
        ed = s * S * (1 + m * c) + m * s * (s * S + c) + m * s * c + 5 * np.abs(d)
    got = forward(fd, dev, a, kind)[1].double().numpy() * 448
    assert np.all(np.abs(got - np.abs(y)) <= ey * EPS)
    for fmt, most in ((0, 448), (1, 57344)):
        got = backward(fd, dev, a, kind, fmt)["dh_s"][0].double().numpy() * most
        live = np.abs(d) > 2.0 ** -99
        assert np.all((np.abs(got - np.abs(d)) <= ed * EPS)[live])
    got = []
    for i in range(0, a.numel(), 1024):  # groups of one row
        part = a[i:i + 1024].contiguous()
        got.append(backward(fd, dev, part, kind, offsets=alone(part.numel())))
    for name, want, err in (("dh_st", d, ed), ("g_st", y, ey)):
        t = np.concatenate([b[name][:, 0].double().numpy() for b in got]) * 448
        live = np.abs(want) > 2.0 ** -99
        assert np.all((np.abs(t - np.abs(want)) <= err * EPS)[live]), name
