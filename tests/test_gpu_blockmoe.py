"""BlockMoE: every stage of a forward and backward pass against 64 bits from what the stage before left, the whole
against the unquantised formula, and the layer captured, on two streams, in micro-batches, with padding and without
tokens.  BlockLinear and BlockExperts with a scratch buffer."""
import numpy as np
import pytest
import torch

import block_reference as br
import moe_reference as mr
import workloads as wl
from helpers import gpu

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


def u8(t):
    return t.detach().cpu().numpy()


def inputs(T, E, H, F, k, gated, name, scale=0.08):
    g = wl.generator(430, name)
    x = wl.normal((T, H), 1.0, g, torch.bfloat16)
    w1 = wl.normal((E, 2 * F if gated else F, H), scale, g, torch.bfloat16)
    w2 = wl.normal((E, H, F), scale, g, torch.bfloat16)
    return x, wl.normal((T, E), 1.5, g, torch.bfloat16), w1, w2, wl.normal((T, H), 1e-3, g, torch.bfloat16)


def make(w1, w2, T, k, act, dev, **kw):
    from fp8_delayed_scaling_gb300.blockmoe import BlockMoE
    return BlockMoE(w1.to(dev), w2.to(dev), T, k, act=act, **kw)


@pytest.mark.parametrize("T,E,H,F,k,act,grad", [(1, 8, 144, 128, 2, 3, 0), (37, 5, 272, 144, 3, 3, 1), (150, 7, 256, 400, 2, 0, 0),
                                                (300, 24, 128, 272, 4, 2, 0), (64, 4, 400, 128, 4, 1, 1)])
def test_stages(T, E, H, F, k, act, grad):
    dev = gpu()
    gated = act >= 2
    W = 2 * F if gated else F
    x, logits, w1, w2, dy = inputs(T, E, H, F, k, gated, "stages%d" % T)
    valid = (torch.arange(T) % 5 != 3) if T > 8 else None
    moe = make(w1, w2, T + 3, k, act, dev, grad_dtype=grad)
    y = moe.forward(x.to(dev), logits.to(dev), valid=None if valid is None else valid.to(dev))
    R = T * k
    r = mr.route(f64(logits), k, None if valid is None else valid.numpy())
    assert np.array_equal(u8(moe.expert), r["expert"]) and np.array_equal(u8(moe.position), r["position"])
    assert np.array_equal(u8(moe.offsets), r["offsets"]) and np.array_equal(u8(moe.counts), r["counts"])
    off, n = r["offsets"].tolist(), int(r["offsets"][-1])
    token = r["token"][:n]
    # dispatch: the tokens' codes in their rows
    xq, xs = br.rows(x.float().numpy(), 0)
    assert np.array_equal(u8(moe._rq)[:R * H].reshape(R, H)[:n], xq[token])
    assert np.array_equal(u8(moe._rs)[:R * br.blocks(H)].reshape(-1, R)[:, :n], xs[:, token])
    X = br.values(xq, 0, xs, 1)[token]
    W1, W2 = (np.stack([(lambda c: br.values(c[0], 0, c[1], 128))(br.weight(m.float().numpy(), 0)) for m in w]) for w in (w1, w2))
    hk = br.values(u8(moe._hq)[:R * W].reshape(R, W)[:n], 0, u8(moe._hs)[:R * br.blocks(W)].reshape(-1, R)[:, :n], 1)
    gk = br.values(u8(moe._gq)[:R * F].reshape(R, F)[:n], 0, u8(moe._gs)[:R * br.blocks(F)].reshape(-1, R)[:, :n], 1)
    ye = f64(moe._ye)[:R * H].reshape(R, H)
    half = {0: 2.0 ** -4, 1: 2.0 ** -3}

    def near(codes, value, err, fmt, axis, what):
        """codes' values against `value` known to err: half a step, the smallest code's, fp32 roundings (see the
        activations' tests); blocks of 128 along axis."""
        amax = np.zeros_like(value)
        for i in range(0, value.shape[axis], 128):
            at = (slice(None), slice(i, i + 128)) if axis else (slice(i, i + 128),)
            amax[at] = (np.abs(value[at]) + err[at]).max(axis, keepdims=True)
        sub = (2.0 ** -10 if fmt == 0 else 2.0 ** -17) / br.MAX[fmt]
        bound = (half[fmt] * (np.abs(value) + err) + sub * amax) * (1 + 2.0 ** -18) + 2.0 ** -21 * np.abs(value) + err + 2.0 ** -100
        assert np.all(np.abs(codes - value) <= bound), what

    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi == lo:
            continue
        h, size = X[lo:hi] @ W1[e].T, np.abs(X[lo:hi]) @ np.abs(W1[e]).T
        eh = br.bound(h, size, H, torch.bfloat16)
        near(hk[lo:hi], h, eh, 0, 1, "h")
        a, b = h[:, :F], h[:, F:]
        v, d, ev, ed = mr.act(a, act)
        ev = ev + 1.2 * eh[:, :F]  # |act'| is at most 1.13
        if gated:
            v, ev = v * b, ev * (np.abs(b) + eh[:, F:]) + np.abs(v) * eh[:, F:] + mr.EPS * np.abs(v * b)
        near(gk[lo:hi], v, ev, 0, 1, "g")
        br.check(torch.from_numpy(ye[lo:hi]).bfloat16(), gk[lo:hi] @ W2[e].T, np.abs(gk[lo:hi]) @ np.abs(W2[e]).T, F, "ye")
    has = r["position"] >= 0
    rows = ye[np.where(has, r["position"], 0)] * has[:, :, None]
    wt = f64(moe.weight)
    want, size = (rows * wt[:, :, None]).sum(1), np.abs(rows * wt[:, :, None]).sum(1)
    assert np.all(np.abs(f64(y) - want) <= 2.0 ** -8 * np.abs(want) * 1.01 + k * mr.EPS * size + 1e-30)
    if valid is not None:
        assert torch.all(y[~valid.to(dev)] == 0)
    # backward
    dloss = torch.full((1,), 0.5, device=dev)
    ye_t = moe._ye[:R * H].clone()
    dx, dlogits, dw1, dw2 = moe.backward(dy.to(dev), dloss)
    D = f64(dy)
    dye = torch.zeros((R, H), dtype=torch.bfloat16)
    t, j = np.nonzero(has)
    dye[r["position"][t, j]] = (dy.float()[t] * moe.weight.cpu()[t, j][:, None]).bfloat16()
    dye = dye[:n]
    dq, ds = br.rows(dye.float().numpy(), grad)
    assert np.array_equal(u8(moe.dye8.row_q)[:n], dq)
    dyek = br.values(dq, grad, ds, 1)
    dweight = (rows * D[:, None]).sum(2)
    assert np.all(np.abs(f64(moe._dweight)[:R].reshape(T, k) - dweight) <= H * mr.EPS * np.abs(rows * D[:, None]).sum(2) + 1e-30)
    dg = f64(moe._h)[:R * F].reshape(R, F)[:n]
    dhk = br.values(u8(moe._dhq)[:R * W].reshape(R, W)[:n], grad, u8(moe._dhs)[:R * br.blocks(W)].reshape(-1, R)[:, :n], 1)
    P = moe._dht.numel() // W if T == moe.tokens else (R + 127 * min(E, R)) // 128 * 128
    cols = lambda q, s, c, f: br.values(u8(q)[:P * c].reshape(c, P), f, u8(s)[:P // 128 * c].reshape(-1, c), 1)  # noqa: E731
    xt, gt, dht = cols(moe._xt, moe._xts, H, 0), cols(moe._gt, moe._gts, F, 0), cols(moe._dht, moe._dhts, W, grad)
    dyet = br.values(u8(moe.dye8.col_q), grad, u8(moe.dye8.col_s), 1)
    at = 0
    dxr = np.zeros((n, H))
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        c = slice(at, at + hi - lo)
        at += br.blocks(hi - lo) * 128
        if hi == lo:
            assert torch.all(dw1[e] == 0) and torch.all(dw2[e] == 0)
            continue
        br.check(torch.from_numpy(dg[lo:hi]).bfloat16(), dyek[lo:hi] @ W2[e], np.abs(dyek[lo:hi]) @ np.abs(W2[e]), H, "dg")
        a, b = hk[lo:hi, :F].astype(np.float32).astype(np.float64), hk[lo:hi, F:]
        v, d, ev, ed = mr.act(a, act)
        ev, ed = ev + mr.EPS * np.abs(a) * 1.2, ed + mr.EPS * np.abs(a)  # the decoded value is rounded to fp32
        G = dg[lo:hi]
        if gated:
            dh = np.concatenate([G * b * d, G * v], 1)
            edh = np.concatenate([np.abs(G * b) * (ed + 4 * mr.EPS), np.abs(G) * (ev + mr.EPS * np.abs(v))], 1)
            v, ev = v * b, (ev + 2 * mr.EPS * np.abs(v)) * np.abs(b)
        else:
            dh, edh = G * d, np.abs(G) * (ed + mr.EPS)
        near(dhk[lo:hi], dh, edh, grad, 1, "dh")
        near(dht[:, c].T, dh, edh, grad, 0, "dh transposed")
        near(gt[:, c].T, v, ev, 0, 0, "g transposed")
        near(xt[:, c].T, X[lo:hi], mr.EPS * np.abs(X[lo:hi]), 0, 0, "x transposed")
        br.check(dw2[e], dyet[:, c] @ gt[:, c].T, np.abs(dyet[:, c]) @ np.abs(gt[:, c]).T, hi - lo, "dw2")
        br.check(dw1[e], dht[:, c] @ xt[:, c].T, np.abs(dht[:, c]) @ np.abs(xt[:, c]).T, hi - lo, "dw1")
        dxr[lo:hi] = f64(moe._ye)[:R * H].reshape(R, H)[lo:hi]
        br.check(torch.from_numpy(dxr[lo:hi]).bfloat16(), dhk[lo:hi] @ W1[e], np.abs(dhk[lo:hi]) @ np.abs(W1[e]), W, "dx rows")
    back = dxr[np.where(has, r["position"], 0)] * has[:, :, None]
    assert np.all(np.abs(f64(dx) - back.sum(1)) <= 2.0 ** -8 * np.abs(back.sum(1)) * 1.01 + k * mr.EPS * np.abs(back).sum(1) + 1e-30)
    dl, size = mr.route_grad(r, f64(moe._dweight)[:R].reshape(T, k), 0.5)
    assert np.all(np.abs(f64(dlogits) - dl) <= 4 * mr.route_error(f64(logits), r)[:, None] * size + 2.0 ** -8 * 1.01 * np.abs(dl) + 1e-30)
    assert not torch.equal(ye_t, moe._ye[:R * H])  # its rows were used again: a second backward is refused
    with pytest.raises(RuntimeError):
        moe.backward(dy.to(dev))


def _whole(x, logits, w1, w2, k, act, dy, dloss):
    """y, dx, dlogits, dw1, dw2 in fp64 by torch's differentiation of the unquantised formula."""
    x, l, w1, w2 = (t.double().requires_grad_() for t in (x, logits, w1, w2))
    p = torch.softmax(l, 1)
    idx = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, idx)
    w = w / w.sum(1, keepdim=True)
    F, y = w2.shape[2], 0
    f = (lambda a: 0.5 * a * torch.special.erfc(-a / 2 ** 0.5)) if act in (0, 2) else (lambda a: a * torch.sigmoid(a))
    for j in range(k):
        h = torch.einsum("th,twh->tw", x, w1[idx[:, j]])
        g = f(h[:, :F]) * h[:, F:] if act >= 2 else f(h)
        y = y + w[:, j, None] * torch.einsum("tf,thf->th", g, w2[idx[:, j]])
    E, T = l.shape[1], l.shape[0]
    counts = torch.bincount(idx.reshape(-1), minlength=E).double()
    loss = E * ((counts / (T * k)) * (p.sum(0) / T)).sum()
    ((y * dy.double()).sum() + dloss * loss).backward()
    return (y.detach(), x.grad, l.grad, w1.grad, w2.grad), loss.detach()


@pytest.mark.parametrize("act", range(4))
def test_whole_layer_against_the_unquantised_formula(act):
    """Each product's operands are off by half a step (e4m3: 2^-4 of a value at most, of random sign), so a result that goes
    through n quantised operands is off by less than n 2^-4 of its norm: two operands each for h and ye, two more for dg
    and dx or a weight's gradient; dlogits follows from ye and dy."""
    dev = gpu()
    T, E, H, F, k = 200, 6, 256, 256, 2
    x, logits, w1, w2, dy = inputs(T, E, H, F, k, act >= 2, "whole")
    moe = make(w1, w2, T, k, act, dev)
    y = moe.forward(x.to(dev), logits.to(dev)).clone()
    got = (y,) + moe.backward(dy.to(dev), torch.full((1,), 0.25, device=dev))
    want, loss = _whole(x, logits, w1, w2, k, act, dy, 0.25)
    assert abs(float(moe.loss) - float(loss)) <= 1e-5 * float(loss)
    for n, (a, b) in zip((4, 8, 4, 8, 8), zip(got, want)):
        assert (a.double().cpu() - b).norm() <= n * 2.0 ** -4 * b.norm()


def test_captured_and_replayed_beside_an_eager_layer():
    dev = gpu()
    T, E, H, F, k = 160, 6, 256, 272, 2
    x, logits, w1, w2, dy = (t.to(dev) for t in inputs(T, E, H, F, k, True, "graph"))
    moe, ref = make(w1, w2, T, k, 3, dev), make(w1, w2, T, k, 3, dev)
    xs, ls, ds, valid = x.clone(), logits.clone(), dy.clone(), torch.ones(T, dtype=torch.bool, device=dev)
    dloss = torch.full((1,), 0.1, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.forward(xs, ls, valid=valid)
        moe.backward(ds, dloss)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = moe.forward(xs, ls, valid=valid)
            out = moe.backward(ds, dloss)
    for i in range(3):
        xs.copy_(torch.roll(x, i, 0)), ls.copy_(torch.roll(logits, i, 1)), ds.copy_(torch.roll(dy, i, 1))
        valid.copy_(torch.arange(T, device=dev) < T - 40 * i)
        ref.forward(xs, ls, valid=valid)
        graph.replay()
        want = ref.backward(ds, dloss)
        torch.cuda.synchronize()
        assert torch.equal(y, ref._y[:T * H].view(T, H)) and all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams_and_every_size_of_batch():
    dev = gpu()
    T, E, H, F, k = 120, 4, 128, 144, 2
    x, logits, w1, w2, dy = (t.to(dev) for t in inputs(T, E, H, F, k, True, "streams"))
    ref = make(w1, w2, T, k, 3, dev)
    torch.cuda.synchronize()
    layers, streams = [make(w1, w2, T, k, 3, dev) for _ in range(2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for n in (T, 1, 77, 0):
        outs = []
        for lay, st in zip(layers, streams):
            y = lay.forward(x[:n], logits[:n], stream=st)
            outs.append((y,) + lay.backward(dy[:n], stream=st))
        want = (ref.forward(x[:n], logits[:n]),) + ref.backward(dy[:n])
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, want)), n
        assert want[0].shape == (n, H) and (n or float(ref.loss) == 0)


def test_micro_batches_and_serving():
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    T, E, H, F, k = 64, 4, 128, 256, 2
    x, logits, w1, w2, dy = (t.to(dev) for t in inputs(T, E, H, F, k, True, "micro"))
    moe, ref = make(w1, w2, T, k, 3, dev), make(w1, w2, T, k, 3, dev)
    with pytest.raises(RuntimeError):
        moe.forward(x, logits, is_first_microbatch=False)
    moe.forward(x, logits, is_first_microbatch=True)
    n0 = fd.fp8dl_kernel_launches()
    y = moe.forward(x, logits, is_first_microbatch=False, need_backward=False)
    launched = fd.fp8dl_kernel_launches() - n0
    assert launched <= 7  # route (two at most), dispatch, two products, activation, combination
    assert torch.equal(y, ref.forward(x, logits))
    with pytest.raises(RuntimeError):
        moe.backward(dy)
    moe.forward(x, logits, is_first_microbatch=False)
    with pytest.raises(ValueError):
        moe.backward(dy[:5])
    with pytest.raises(ValueError):
        moe.forward(torch.cat([x, x]), torch.cat([logits, logits]))
    assert all(torch.equal(a, b) for a, b in zip(moe.backward(dy), ref.backward(dy)))


@pytest.mark.parametrize("rows", [1, 128, 300])
def test_linear_and_experts_with_scratch(rows):
    """Layers that keep row-wise codes and share one scratch buffer: all but the weight's gradient as without it, the gradient
    from the codes that the row-wise ones give."""
    from fp8_delayed_scaling_gb300.blocklinear import BlockExperts, BlockLinear, block_scratch_size
    dev = gpu()
    n, k, off = 272, 400, [0, rows // 3, rows // 3, rows]
    g = wl.generator(431, "scratch%d" % rows)
    x, dy = wl.student_t3((rows, k), 0.5, g), wl.normal((rows, n), 1e-3, g, torch.bfloat16)
    w, w3 = wl.normal((n, k), 0.02, g, torch.bfloat16), wl.normal((3, n, k), 0.02, g, torch.bfloat16)
    scratch = torch.full((max(block_scratch_size(300, k), block_scratch_size(300, k, 3)),), 0xEE, dtype=torch.uint8, device=dev)
    plain, lean = BlockLinear(w.to(dev), None, 300), BlockLinear(w.to(dev), None, 300, scratch=scratch)
    eplain, elean = BlockExperts(w3.to(dev), 300), BlockExperts(w3.to(dev), 300, scratch=scratch)
    o = torch.tensor(off, dtype=torch.int32, device=dev)
    y, ey = lean.forward(x.to(dev)), elean.forward(x.to(dev), o)
    assert torch.all(scratch == 0xEE)  # the forward passes leave it alone
    assert torch.equal(y, plain.forward(x.to(dev))) and torch.equal(ey, eplain.forward(x.to(dev), o))
    q, s = br.rows(x.float().numpy(), 0)
    kept = (torch.from_numpy(q).view(torch.float8_e4m3fn).float().numpy() * np.repeat(s.T, 128, 1)[:, :k]).astype(np.float32)
    dx, dw, _ = lean.backward(dy.to(dev))
    pdx, pdw, _ = plain.backward(dy.to(dev))
    assert torch.equal(dx, pdx)
    cols = lambda v, of: (lambda c: br.values(c[0], 0, c[1], 1))(br.cols(v, 0, of))  # noqa: E731
    a, b = cols(dy.float().numpy(), None), cols(kept, None)
    br.check(dw, a @ b.T, np.abs(a) @ np.abs(b).T, rows, "dw")
    edx, edw = elean.backward(dy.to(dev))
    assert torch.equal(edx, eplain.backward(dy.to(dev))[0])
    a, b, at = cols(dy.float().numpy(), off), cols(kept, off), 0
    for e in range(3):
        m = off[e + 1] - off[e]
        c = slice(at, at + m)
        at += br.blocks(m) * 128
        br.check(edw[e], a[:, c] @ b[:, c].T, np.abs(a[:, c]) @ np.abs(b[:, c]).T, max(m, 1), "experts' dw")
    assert torch.equal(lean.forward(x.to(dev)), plain.forward(x.to(dev)))  # micro-batch after micro-batch
    with pytest.raises(ValueError):
        BlockLinear(w.to(dev), None, 300, scratch=scratch[:100])
    with pytest.raises(ValueError):
        BlockLinear(w.to(dev), None, 300, scratch=scratch[1:])
