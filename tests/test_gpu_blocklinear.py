"""BlockLinear and BlockExperts: a whole forward and backward pass against plain numpy, from the
same codes (within the product bound) and from the unquantised formula (within the rounding of
the codes); captured into a graph, on another stream, with micro-batches and single tokens."""
import numpy as np
import pytest
import torch

import block_reference as br
import workloads as wl
from helpers import gpu

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.detach().double().cpu().numpy()


def _code_error(x, fmt, axis):
    """How far codes may be from x: half a step of the value (e4m3 2^-4, e5m2 2^-3 of it) or half the smallest code's
    step, in units of the stored factor; `axis` None: 128 x 128 blocks, else blocks of 128 along it.  The scaled value,
    the scale and its reciprocal are each rounded to fp32 first: 2^-18 covers those."""
    half, sub = (2.0 ** -4, 2.0 ** -10) if fmt == 0 else (2.0 ** -3, 2.0 ** -17)
    amax = np.zeros_like(x)
    for i in range(0, x.shape[0], 128 if axis != 1 else 1):
        for j in range(0, x.shape[1], 128 if axis != 0 else 1):
            at = (slice(i, i + (128 if axis != 1 else 1)), slice(j, j + (128 if axis != 0 else 1)))
            amax[at] = np.abs(x[at]).max()
    return (half * np.abs(x) + sub * amax / br.MAX[fmt]) * (1 + 2.0 ** -18) + 2.0 ** -22 * np.abs(x)


def _product_error(a, b, ea, eb, dtype):
    """|Q(a) Q(b)^T - a b^T| at most, with the product's own error and the output's rounding."""
    e = np.abs(a) @ eb.T + ea @ np.abs(b).T + ea @ eb.T
    return e + br.bound(np.abs(a @ b.T) + e, np.abs(a) @ np.abs(b).T + e, a.shape[1], dtype)


def _inputs(rows, n, k, name, lead=()):
    g = wl.generator(310, name)
    x = wl.student_t3((rows, k), 0.5, g)
    w = wl.normal(lead + (n, k), 0.02, g, torch.bfloat16)
    dy = wl.normal((rows, n), 1e-3, g, torch.bfloat16)
    return x, w, dy


@pytest.mark.parametrize("grad", [0, 1])
@pytest.mark.parametrize("rows,n,k", [(1, 144, 272), (37, 400, 528), (300, 272, 640)])
def test_linear_step(rows, n, k, grad):
    from fp8_delayed_scaling_gb300.blocklinear import BlockLinear
    dev = gpu()
    x, w, dy = _inputs(rows, n, k, "step%d" % rows)
    b = wl.normal((n,), 0.1, wl.generator(311, "b"), torch.bfloat16)
    lin = BlockLinear(w.to(dev), b.to(dev), 512, grad_dtype=grad)
    y = lin.forward(x.to(dev))
    dx, dw, db = lin.backward(dy.to(dev))
    X, W, G, B = _f64(x), _f64(w), _f64(dy), _f64(b)
    # the same codes
    xq, wq = br.values(*_rows(x, 0)), br.values(*_blocks(w), 128)
    gq = br.values(*_rows(dy, grad))
    br.check(y, xq @ wq.T + B, np.abs(xq) @ np.abs(wq).T + np.abs(B), k, "y")
    br.check(dx, gq @ wq, np.abs(gq) @ np.abs(wq), n, "dx")
    gt, xt = br.values(*_cols(dy, grad)), br.values(*_cols(x, 0))
    br.check(dw, gt @ xt.T, np.abs(gt) @ np.abs(xt).T, rows, "dw")
    assert np.all(np.abs(_f64(db) - G.sum(0)) <= rows * 2.0 ** -24 * np.abs(G).sum(0))
    # the formula, within the codes' rounding
    ew = _code_error(W, 0, None)
    ey = _product_error(X, W, _code_error(X, 0, 1), ew, y.dtype) + 2.0 ** -8 * np.abs(B)
    edx = _product_error(G, W.T, _code_error(G, grad, 1), ew.T, dx.dtype)
    edw = _product_error(G.T, X.T, _code_error(G, grad, 0).T, _code_error(X, 0, 0).T, dw.dtype)
    assert np.all(np.abs(_f64(y) - X @ W.T - B) <= ey)
    assert np.all(np.abs(_f64(dx) - G @ W) <= edx)
    assert np.all(np.abs(_f64(dw) - G.T @ X) <= edw)
    # differences of the loss sum(G * (X W^T + b)) along random directions
    loss = lambda X, W, B: (G * (X @ W.T + B)).sum()  # noqa: E731
    rng = np.random.default_rng(3)
    for arg, grad_t, err in ((0, _f64(dx), edx), (1, _f64(dw), edw)):
        v = rng.standard_normal((X, W)[arg].shape)
        h = 1e-3
        at = [X, W, B]
        plus, minus = list(at), list(at)
        plus[arg], minus[arg] = at[arg] + h * v, at[arg] - h * v
        d = (loss(*plus) - loss(*minus)) / (2 * h)
        assert abs(d - (grad_t * v).sum()) <= (err * np.abs(v)).sum() + 1e-9 * abs(d)


def _rows(t, fmt):
    q, s = br.rows(t.float().numpy(), fmt)
    return q, fmt, s, 1


def _cols(t, fmt):
    q, s, _ = br.cols(t.float().numpy(), fmt)
    return q, fmt, s, 1


def _blocks(t):
    q, s = br.weight(t.float().numpy(), 0)
    return q, 0, s


@pytest.mark.parametrize("off,rows", [([0, 1, 1, 4], 6), ([0, 0, 150, 150], 150), ([2, 40, 180, 500], 513)],
                         ids=["decode", "one busy", "ragged"])
def test_experts_step(off, rows):
    from fp8_delayed_scaling_gb300.blocklinear import BlockExperts
    dev = gpu()
    G, n, k = len(off) - 1, 272, 400
    x, w, dy = _inputs(rows, n, k, "experts%d" % rows, (G,))
    o = torch.tensor(off, dtype=torch.int32, device=dev)
    ex = BlockExperts(w.to(dev), 600, grad_dtype=1)
    ex._y.fill_(7.0)
    ex._dx.fill_(7.0)
    y = ex.forward(x.to(dev), o)
    dx, dw = ex.backward(dy.to(dev))
    X, W, D = _f64(x), _f64(w), _f64(dy)
    for t in (y, dx):
        assert torch.all(t[:off[0]] == 7.0) and torch.all(t[off[-1]:] == 7.0)
    for g, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        if lo == hi:
            assert torch.all(dw[g] == 0)
            continue
        a, b, c = X[lo:hi], W[g], D[lo:hi]
        ew = _code_error(b, 0, None)
        assert np.all(np.abs(_f64(y[lo:hi]) - a @ b.T) <= _product_error(a, b, _code_error(a, 0, 1), ew, y.dtype))
        assert np.all(np.abs(_f64(dx[lo:hi]) - c @ b) <= _product_error(c, b.T, _code_error(c, 1, 1), ew.T, dx.dtype))
        assert np.all(np.abs(_f64(dw[g]) - c.T @ a) <= _product_error(
            c.T, a.T, _code_error(c, 1, 0).T, _code_error(a, 0, 0).T, dw.dtype))


def test_experts_in_two_layers_match_a_loop_over_linears():
    """Two expert layers with an activation between them, forward and backward, as a loop of BlockLinear over the
    experts gives them: the same bits, since every block has the same values."""
    from fp8_delayed_scaling_gb300.blocklinear import BlockExperts, BlockLinear
    dev = gpu()
    off, h, f = [0, 130, 130, 300, 301], 256, 384
    g = wl.generator(320, "two")
    x = wl.normal((off[-1], h), 1.0, g, torch.bfloat16).to(dev)
    w1, w2 = wl.normal((4, f, h), 0.05, g, torch.bfloat16).to(dev), wl.normal((4, h, f), 0.05, g, torch.bfloat16).to(dev)
    dy = wl.normal((off[-1], h), 1e-3, g, torch.bfloat16).to(dev)
    o = torch.tensor(off, dtype=torch.int32, device=dev)
    e1, e2 = BlockExperts(w1, 301), BlockExperts(w2, 301)
    a = e1.forward(x, o)
    y = e2.forward(torch.relu(a), o).clone()
    da, dw2 = e2.backward(dy)
    dx, dw1 = e1.backward(da * (a > 0))
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        if lo == hi:
            continue
        l1, l2 = BlockLinear(w1[e], None, hi - lo), BlockLinear(w2[e], None, hi - lo)
        b = l1.forward(x[lo:hi])
        yb = l2.forward(torch.relu(b))
        db, dw2b, _ = l2.backward(dy[lo:hi].contiguous())
        dxb, dw1b, _ = l1.backward(db * (b > 0))
        tol = 2.0 ** -7  # the layers may split K differently: a few fp32 roundings, which move a bf16 by one step
        for got, ref in ((y[lo:hi], yb), (dw2[e], dw2b), (dx[lo:hi], dxb), (dw1[e], dw1b)):
            r = ref.float()
            # where the codes in between moved by a step the sums move with them: those stay small against the whole
            assert (got.float() - r).norm() <= tol * r.norm()


def test_micro_batches_reuse_the_weight():
    import fp8_delayed_scaling_gb300 as fd
    from fp8_delayed_scaling_gb300.blocklinear import BlockLinear
    dev = gpu()
    x, w, dy = _inputs(128, 256, 256, "micro")
    x, w, dy = x.to(dev), w.to(dev), dy.to(dev)
    lin, ref = BlockLinear(w, None, 128), BlockLinear(w, None, 128)
    lin.forward(x, is_first_microbatch=True)
    n0 = fd.fp8dl_kernel_launches()
    y = lin.forward(x, is_first_microbatch=False)
    assert fd.fp8dl_kernel_launches() - n0 == 2  # the input's quantisation and the product
    assert torch.equal(y, ref.forward(x))
    out, want = lin.backward(dy), ref.backward(dy)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    n0 = fd.fp8dl_kernel_launches()
    ref.backward(dy)
    assert fd.fp8dl_kernel_launches() - n0 == 3
    y1 = lin.forward(x[:1], is_first_microbatch=False, need_backward=False)  # one token against the kept weight
    assert y1.shape == (1, 256)
    with pytest.raises(RuntimeError):
        lin.backward(dy[:1])
    q, s = br.rows(x[:1].float().cpu().numpy(), 0)
    wq = br.values(*_blocks(w.cpu()), 128)
    xq = br.values(q, 0, s, 1)
    br.check(y1, xq @ wq.T, np.abs(xq) @ np.abs(wq).T, 256, "one token")


def test_no_rows():
    from fp8_delayed_scaling_gb300.blocklinear import BlockExperts, BlockLinear
    dev = gpu()
    x, dy = torch.zeros((0, 256), dtype=torch.bfloat16, device=dev), torch.zeros((0, 128), dtype=torch.bfloat16, device=dev)
    w = torch.ones((3, 128, 256), dtype=torch.bfloat16, device=dev)
    lin = BlockLinear(w[0], torch.ones(128, dtype=torch.bfloat16, device=dev), 16)
    lin.dw.fill_(7.0), lin.db.fill_(7.0)
    assert lin.forward(x).shape == (0, 128)
    dx, dw, db = lin.backward(dy)
    assert dx.shape == (0, 256) and torch.all(dw == 0) and torch.all(db == 0)
    ex = BlockExperts(w, 16)
    ex.dw.fill_(7.0)
    o = torch.zeros(4, dtype=torch.int32, device=dev)
    assert ex.forward(x, o).shape == (0, 128)
    dx, dw = ex.backward(dy)
    assert dx.shape == (0, 256) and torch.all(dw == 0)


def test_step_captured_and_replayed_with_other_groups():
    """A captured expert step replays on new inputs and new offsets, while an eager layer works beside it."""
    from fp8_delayed_scaling_gb300.blocklinear import BlockExperts
    dev = gpu()
    G, n, k, rows = 5, 272, 256, 200
    x, w, dy = _inputs(rows, n, k, "graph", (G,))
    x, w, dy = x.to(dev), w.to(dev), dy.to(dev)
    offs = [[0, 50, 60, 60, 130, 200], [0, 0, 0, 200, 200, 200], [0, 1, 2, 3, 4, 5]]
    o = torch.tensor(offs[0], dtype=torch.int32, device=dev)
    xs, dys = x.clone(), dy.clone()
    ex, ref = BlockExperts(w, rows), BlockExperts(w, rows)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ex.forward(xs, o)
        ex.backward(dys)  # warm up
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = ex.forward(xs, o)
            dx, dw = ex.backward(dys)
    for i, off in enumerate(offs):
        o.copy_(torch.tensor(off, dtype=torch.int32))
        xs.copy_(torch.roll(x, i, 0))
        dys.copy_(torch.roll(dy, i, 1))
        for t in (y, dx):
            t.fill_(3.0)
        graph.replay()
        ref._y.fill_(3.0), ref._dx.fill_(3.0)
        ry = ref.forward(xs, o)
        rdx, rdw = ref.backward(dys)
        torch.cuda.synchronize()
        assert torch.equal(y, ry) and torch.equal(dx, rdx) and torch.equal(dw, rdw)


def test_two_layers_on_two_streams():
    from fp8_delayed_scaling_gb300.blocklinear import BlockLinear
    dev = gpu()
    x, w, dy = _inputs(512, 768, 1024, "streams")
    x, w, dy = x.to(dev), w.to(dev), dy.to(dev)
    want = BlockLinear(w, None, 512)
    wy = want.forward(x).clone()
    wdx, wdw, _ = want.backward(dy)
    torch.cuda.synchronize()
    layers = [BlockLinear(w, None, 512) for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs = []
        for lay, st in zip(layers, streams):
            y = lay.forward(x, stream=st)
            outs.append((y,) + lay.backward(dy, stream=st)[:2])
    torch.cuda.synchronize()
    for y, dx, dw in outs:
        assert torch.equal(y, wy) and torch.equal(dx, wdx) and torch.equal(dw, wdw)
