"""fp8_block_dispatch, moe_combine and moe_combine_bwd: codes and the gradient of the rows bit by bit, sums
against 64 bits."""
import numpy as np
import pytest
import torch

import block_reference as br
import moe_reference as mr
import workloads as wl
from helpers import gpu

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 16, 1), (1, 6, 4096, 6), (3, 2, 144, 9), (37, 6, 1040, 300), (129, 4, 272, 516), (200, 8, 1024, 1700), (70, 32, 400, 2240),
         (515, 2, 2064, 1030)]


def positions(T, k, R, name):
    """Distinct rows of R, some of them out of range (negative and behind the end) or not there."""
    g = wl.generator(410, name)
    pos = torch.randperm(max(R, T * k), generator=g)[:T * k].view(T, k).int()
    drop = torch.rand((T, k), generator=g)
    pos[drop < 0.1] = -1
    pos[(drop > 0.1) & (drop < 0.13)] = -(1 << 31)
    pos[(drop > 0.13) & (drop < 0.16)] = R
    pos[(drop > 0.16) & (drop < 0.19)] = (1 << 31) - 1
    return pos


@pytest.mark.parametrize("T,k,C,R", SIZES)
@pytest.mark.parametrize("dtype,fmt", [(torch.bfloat16, 0), (torch.float32, 1)])
def test_dispatch(T, k, C, R, dtype, fmt):
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    x = wl.student_t3((T, C), 0.5, wl.generator(411, "x"), dtype)
    if T > 2:
        x[0, :7], x[1, 3], x[1, 5] = 0.0, float("inf"), float("nan")
        x[2] = 0.0
    pos = positions(T, k, R, "d%d" % T)
    want, ws = br.rows(x.float().numpy(), fmt)
    blocks = br.blocks(C)
    for keep in (True, False):
        rq, rs = torch.full((R, C), 0xAB, dtype=torch.uint8, device=dev), torch.full((blocks, R), -7.0, device=dev)
        q, s = torch.full((T, C), 0xAB, dtype=torch.uint8, device=dev), torch.full((blocks, T), -7.0, device=dev)
        fd.fp8_block_dispatch(x.to(dev), fmt, pos.to(dev), rq, rs, q=q if keep else None, s=s if keep else None)
        eq, es = np.full((R, C), 0xAB, np.uint8), np.full((blocks, R), -7.0, np.float32)
        for t in range(T):
            for p in pos[t].tolist():
                if 0 <= p < R:
                    eq[p], es[:, p] = want[t], ws[:, t]
        got = rq.cpu().numpy()
        nan = torch.from_numpy(eq).view(br.F8[fmt]).float().isnan().numpy()
        assert np.array_equal(got[~nan], eq[~nan]) and torch.from_numpy(got).view(br.F8[fmt]).float().isnan().numpy()[nan].all()
        assert np.array_equal(rs.cpu().numpy(), es)
        if keep:
            fq, fs = torch.zeros_like(q), torch.zeros_like(s)
            fd.fp8_block_quantize(x.to(dev), fmt, row_q=fq, row_s=fs)
            assert torch.equal(q, fq) and torch.equal(s, fs)
        else:
            assert torch.all(q == 0xAB) and torch.all(s == -7.0)


@pytest.mark.parametrize("T,k,C,R", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_combine_and_gradient(T, k, C, R, dtype):
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    y = wl.normal((R, C), 1.0, wl.generator(412, "y"), dtype)
    w = wl.normal((T, k), 1.0, wl.generator(412, "w"), torch.float32)
    pos = positions(T, k, R, "c%d" % T)
    ok = (pos >= 0) & (pos < R)
    idx = torch.where(ok, pos, 0).long()
    Y = y.double()[idx] * ok[:, :, None]
    half = torch.finfo(dtype).eps / 2
    for weight in (w, None):
        out = torch.full((T, C), 9.0, dtype=dtype, device=dev)
        fd.moe_combine(y.to(dev), pos.to(dev), out, weight=None if weight is None else w.to(dev))
        W = w.double() if weight is not None else torch.ones((T, k), dtype=torch.double)
        want, size = (Y * W[:, :, None]).sum(1), (Y * W[:, :, None]).abs().sum(1)
        assert torch.all((out.double().cpu() - want).abs() <= half * want.abs() * 1.01 + k * mr.EPS * size + 2.0 ** -140)
    dout = wl.normal((T, C), 1e-3, wl.generator(412, "d"), dtype)
    dwant = (Y * dout.double()[:, None]).sum(2)
    dsize = (Y * dout.double()[:, None]).abs().sum(2)
    rows = torch.full((R, C), -7.0, dtype=dtype)
    rows[idx[ok]] = (dout.float()[:, None] * w[:, :, None]).to(dtype)[ok]
    for parts in ("both", "dy", "dweight"):
        dy, dw = torch.full((R, C), -7.0, dtype=dtype, device=dev), torch.full((T, k), 9.0, device=dev)
        fd.moe_combine_bwd(dout.to(dev), None if parts == "dy" else y.to(dev), pos.to(dev), None if parts == "dweight" else w.to(dev),
                           dy=None if parts == "dweight" else dy, dweight=None if parts == "dy" else dw)
        if parts != "dweight":
            assert torch.equal(dy.cpu(), rows)  # one product in fp32, one rounding
        if parts != "dy":
            assert torch.all((dw.double().cpu() - dwant).abs() <= C * mr.EPS * dsize + 2.0 ** -140)
            assert torch.all(dw.cpu()[~ok] == 0)


def test_no_tokens_and_no_rows():
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    z = lambda *s, d=torch.float32: torch.zeros(s, dtype=d, device=dev)  # noqa: E731
    pos = z(0, 2, d=torch.int32)
    fd.fp8_block_dispatch(z(0, 64), 0, pos, z(4, 64, d=torch.uint8), z(1, 4))
    fd.moe_combine(z(4, 64), pos, z(0, 64), weight=z(0, 2))
    fd.moe_combine_bwd(z(0, 64), z(4, 64), pos, z(0, 2), dy=z(4, 64), dweight=z(0, 2))
    some, out, dw = torch.full((3, 2), 0, dtype=torch.int32, device=dev), torch.full((3, 64), 5.0, device=dev), torch.full((3, 2), 5.0, device=dev)
    fd.moe_combine(z(0, 64), some, out)                          # no row to name: zeros
    fd.moe_combine_bwd(out, z(0, 64), some, dw, dy=z(0, 64), dweight=dw)
    q, s = torch.full((3, 64), 9, dtype=torch.uint8, device=dev), z(1, 3)
    fd.fp8_block_dispatch(out, 0, some, z(0, 64, d=torch.uint8), z(1, 0), q=q, s=s)
    assert torch.all(out == 0) and torch.all(dw == 0) and torch.all(q == 0) and torch.all(s == 1)


def test_values_that_are_not_finite():
    """An infinity or NaN reaches the tokens that take its row, and no others; weight 0 does not hide it."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    y = torch.ones((6, 128), device=dev)
    y[2, 5], y[4, 100] = float("inf"), float("nan")
    pos = torch.tensor([[0, 1], [2, 3], [4, 5], [1, -1]], dtype=torch.int32, device=dev)
    w = torch.tensor([[1.0, 1], [1, 1], [1, 1], [2, float("nan")]], device=dev)  # the NaN weight has no row
    out = torch.zeros((4, 128), device=dev)
    fd.moe_combine(y, pos, out, weight=w)
    assert torch.all(out[0] == 2) and torch.all(out[3] == 2)
    assert torch.isinf(out[1, 5]) and torch.isnan(out[2, 100]) and int(torch.isfinite(out).sum()) == 4 * 128 - 2
