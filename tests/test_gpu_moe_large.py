"""Routing, exchange and 8-bit activations past 2^31 bytes or elements of an operand or a result: every offset is a
64-bit one.  A row, a tile of rows or a token is the same, bit by bit, as in a call for it alone."""
import pytest
import torch

from helpers import gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8, device="cuda")


def _f32(*shape):
    return torch.zeros(shape, device="cuda")


@pytest.mark.parametrize("act", [0, 3])
def test_activation_and_gradient(act):
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    R, C = 65536 + 40, 40960
    W = 2 * C if act >= 2 else C
    g = torch.Generator(device=dev).manual_seed(1)
    h = torch.empty((R, W), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    dg = torch.empty((R, C), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    T = fd.fp8_block_padded_rows(R)
    gq, gs, hq, hs = _u8(R, C), _f32(C // 128, R), _u8(R, W), _f32(W // 128, R)
    fd.fp8_block_act(h, act, 0, gq, gs, h_q=hq, h_s=hs)
    dq, ds, dt, dts, gt, gts = _u8(R, W), _f32(W // 128, R), _u8(W, T), _f32(T // 128, W), _u8(C, T), _f32(T // 128, C)
    fd.fp8_block_dact(dg, hq, 0, hs, act, 0, dh_q=dq, dh_s=ds, dh_qt=dt, dh_st=dts, g_qt=gt, g_st=gts)
    edge = [(1 << 31) // n // 128 for n in (C, W, 2 * W)]  # tiles around element 2^31 (or byte 2^31)
    for tile in sorted({0, 200, T // 128 - 1} | {e + d for e in edge for d in (-1, 0, 1) if 0 <= e + d < T // 128}):
        lo, hi = 128 * tile, min(128 * tile + 128, R)
        m = hi - lo
        a = _u8(m, C), _f32(C // 128, m), _u8(m, W), _f32(W // 128, m)
        fd.fp8_block_act(h[lo:hi], act, 0, a[0], a[1], h_q=a[2], h_s=a[3])
        assert torch.equal(gq[lo:hi], a[0]) and torch.equal(gs[:, lo:hi], a[1]), tile
        assert torch.equal(hq[lo:hi], a[2]) and torch.equal(hs[:, lo:hi], a[3]), tile
        b = _u8(m, W), _f32(W // 128, m), _u8(W, 128), _f32(1, W), _u8(C, 128), _f32(1, C)
        fd.fp8_block_dact(dg[lo:hi], a[2], 0, a[3], act, 0, dh_q=b[0], dh_s=b[1], dh_qt=b[2], dh_st=b[3], g_qt=b[4], g_st=b[5])
        assert torch.equal(dq[lo:hi], b[0]) and torch.equal(ds[:, lo:hi], b[1]), tile
        assert torch.equal(dt[:, lo:lo + 128], b[2]) and torch.equal(dts[tile:tile + 1], b[3]), tile
        assert torch.equal(gt[:, lo:lo + 128], b[4]) and torch.equal(gts[tile:tile + 1], b[5]), tile
    # codes along the rows alone are another kernel's
    dq2, ds2 = _u8(R, W), _f32(W // 128, R)
    fd.fp8_block_dact(dg, hq, 0, hs, act, 0, dh_q=dq2, dh_s=ds2)
    assert torch.equal(dq, dq2) and torch.equal(ds, ds2)


def test_recode():
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    S, R, C = 65600, 70000, 40960
    g = torch.Generator(device=dev).manual_seed(2)
    q = torch.randint(0, 0x78, (S, C), dtype=torch.uint8, device=dev, generator=g)
    s = torch.rand((C // 128, S), device=dev, generator=g) + 0.5
    index = torch.randint(0, S, (R,), dtype=torch.int32, device=dev, generator=g)
    T = fd.fp8_block_padded_rows(R)
    cq, cs = _u8(C, T), _f32(T // 128, C)
    fd.fp8_block_recode(q, 0, s, 0, cq, cs, index=index)
    for tile in (0, 1, T // 256, T // 128 - 2, T // 128 - 1):
        lo, hi = 128 * tile, min(128 * tile + 128, R)
        rows = index[lo:hi].long()
        wq, ws = _u8(C, 128), _f32(1, C)
        fd.fp8_block_recode(q[rows], 0, s[:, rows].contiguous(), 0, wq, ws)
        assert torch.equal(cq[:, lo:lo + 128], wq) and torch.equal(cs[tile:tile + 1], ws), tile


def test_exchange():
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    T, k, C = 9000, 8, 40960
    R = T * k
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.empty((T, C), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    pos = torch.randperm(R, device=dev, generator=g).view(T, k).int()
    w = torch.rand((T, k), device=dev, generator=g)
    rq, rs, q, s = _u8(R, C), _f32(C // 128, R), _u8(T, C), _f32(C // 128, T)
    fd.fp8_block_dispatch(x, 0, pos, rq, rs, q=q, s=s)
    for j in range(k):
        assert torch.equal(rq[pos[:, j].long()], q) and torch.equal(rs[:, pos[:, j].long()], s)
    del rq, q
    y = torch.empty((R, C), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    out, dy, dw = torch.zeros_like(x), torch.zeros_like(y), _f32(T, k)
    fd.moe_combine(y, pos, out, weight=w)
    fd.moe_combine_bwd(x, y, pos, w, dy=dy, dweight=dw)
    small = torch.arange(k, dtype=torch.int32, device=dev).view(1, k)
    last = int((pos == R - 1).nonzero()[0, 0])
    for t in sorted({0, 1, T // 2, T - 1, last}):
        rows = pos[t].long()
        o, d = torch.zeros((1, C), dtype=torch.bfloat16, device=dev), torch.zeros((k, C), dtype=torch.bfloat16, device=dev)
        fd.moe_combine(y[rows], small, o, weight=w[t:t + 1])
        assert torch.equal(out[t:t + 1], o), t
        fd.moe_combine_bwd(x[t:t + 1], y[rows], small, w[t:t + 1], dy=d)
        assert torch.equal(dy[rows], d), t
        want = (x[t].double() * y[rows].double()).sum(1)
        size = (x[t].double() * y[rows].double()).abs().sum(1)
        assert torch.all((dw[t].double() - want).abs() <= (C + 16) * 2.0 ** -24 * size), t


def test_route():
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    T, E, k = (1 << 21) + 77, 1024, 4
    g = torch.Generator(device=dev).manual_seed(4)
    l = torch.empty((T, E), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    i32 = dict(dtype=torch.int32, device=dev)

    def run(l):
        n = l.shape[0]
        b = [torch.zeros((n, k), **i32), _f32(n, k), torch.zeros((n, k), **i32), torch.zeros(n * k, **i32), torch.zeros(E + 1, **i32),
             torch.zeros(E, **i32), _f32(E), _f32(1)]
        fd.moe_route(l, *b[:5], counts=b[5], slope=b[6], loss=b[7], workspace=_u8(fd.moe_route_workspace_size(n, E)))
        return b

    expert, weight, position, token, offsets, counts, slope, loss = run(l)
    flat = torch.arange(T, **i32)[:, None].expand(T, k)
    assert torch.equal(token[position.long()], flat)
    assert torch.equal(torch.bincount(expert.view(-1), minlength=E).int(), counts)
    assert torch.equal(offsets, torch.cat([torch.zeros(1, **i32), counts.cumsum(0).int()]))
    of = torch.searchsorted(offsets.long(), torch.arange(T * k, device=dev), right=True) - 1  # a row's expert
    assert torch.equal(of[position.long()].int(), expert)
    assert torch.all((token[1:] > token[:-1]) | (of[1:] != of[:-1]))  # an expert's rows in the order of their tokens
    d = torch.zeros_like(l)
    dweight, dloss = torch.rand((T, k), device=dev, generator=g), torch.full((1,), 1e4, device=dev)
    fd.moe_route_bwd(l, expert, weight, d, dweight=dweight, slope=slope, dloss=dloss)
    edge = (1 << 31) // E
    rows = torch.tensor([0, 1, edge // 2, edge - 1, edge, edge + 1, T - 2, T - 1], device=dev)
    part = run(l[rows])
    assert torch.equal(part[0], expert[rows]) and torch.equal(part[1], weight[rows])
    pd = torch.zeros((rows.numel(), E), dtype=torch.bfloat16, device=dev)
    fd.moe_route_bwd(l[rows], part[0], part[1], pd, dweight=dweight[rows], slope=slope, dloss=dloss)
    assert torch.equal(pd, d[rows])
    assert abs(float(loss) - 1) < 0.05  # even experts: close to 1
