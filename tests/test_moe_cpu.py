"""Expert routing, token exchange and kept activations without a GPU: the refusals of the C entries and of the
binding (every check comes before the first launch), and the plain reference on cases worked out by hand."""
import numpy as np
import pytest
import torch

import moe_reference as mr


@pytest.fixture(scope="module")
def fd():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_delayed_scaling_gb300
    return fp8_delayed_scaling_gb300


A = 1 << 20  # a fake, 16-byte aligned address: validation fails before any use


def test_routing_entries_refuse_on_the_host(fd):
    L = fd._lib
    need = fd.moe_route_workspace_size(100, 24)
    assert need > 0 and fd.moe_route_workspace_size(0, 24) == 0 and fd.moe_route_workspace_size(100, 1025) == 0
    assert fd.moe_route_workspace_size(1 << 30, 24) == fd.moe_route_workspace_size(160, 24)  # bounded
    route = lambda l=A, dt=1, T=100, E=24, k=4, ex=A, w=A, off=A, slope=A, loss=A, ws=A, wb=need, cnt=None: L.moe_route(  # noqa: E731
        l, dt, T, E, k, None, 1, ex, w, A, A, off, cnt, slope, loss, ws, wb, None)
    assert route(l=None) == fd.ERR_INVALID_ARG
    assert route(dt=2) == fd.ERR_INVALID_ARG
    assert route(E=0) == fd.ERR_INVALID_ARG
    assert route(E=1025) == fd.ERR_INVALID_ARG
    assert route(k=0) == fd.ERR_INVALID_ARG
    assert route(k=25) == fd.ERR_INVALID_ARG           # more choices than experts
    assert route(E=64, k=33, wb=1 << 20) == fd.ERR_INVALID_ARG
    assert route(T=-1) == fd.ERR_SHAPE
    assert route(T=1 << 31, k=1) == fd.ERR_SHAPE
    assert route(T=1 << 29, k=4) == fd.ERR_SHAPE       # 2^31 rows
    assert route(ex=None) == fd.ERR_INVALID_ARG
    assert route(off=None, T=0) == fd.ERR_INVALID_ARG  # written even without tokens
    assert route(slope=None) == fd.ERR_INVALID_ARG     # a loss without its slope
    assert route(l=A + 8) == fd.ERR_ALIGN
    assert route(w=A + 2) == fd.ERR_ALIGN
    assert route(cnt=A + 1) == fd.ERR_ALIGN
    assert route(ws=None) == fd.ERR_WORKSPACE
    assert route(wb=need - 1) == fd.ERR_WORKSPACE
    assert route(ws=A + 8) == fd.ERR_ALIGN
    back = lambda l=A, T=100, k=4, ex=A, slope=A, dl=A, out=A: L.moe_route_bwd(  # noqa: E731
        l, 1, T, 24, k, 1, ex, A, A, slope, dl, out, None)
    assert back(l=None) == fd.ERR_INVALID_ARG
    assert back(ex=None) == fd.ERR_INVALID_ARG
    assert back(out=None) == fd.ERR_INVALID_ARG
    assert back(slope=None) == fd.ERR_INVALID_ARG      # a loss gradient without the slope
    assert back(k=40) == fd.ERR_INVALID_ARG
    assert back(T=1 << 30) == fd.ERR_SHAPE
    assert back(out=A + 8) == fd.ERR_ALIGN
    assert back(dl=A + 2) == fd.ERR_ALIGN


def test_exchange_entries_refuse_on_the_host(fd):
    L = fd._lib
    send = lambda x=A, dt=1, T=10, C=256, fmt=0, pos=A, k=2, R=20, rq=A, rs=A, q=None, s=None: L.fp8_block_dispatch(  # noqa: E731
        x, dt, T, C, fmt, pos, k, R, rq, rs, q, s, None)
    assert send(x=None) == fd.ERR_INVALID_ARG
    assert send(dt=3) == fd.ERR_INVALID_ARG
    assert send(fmt=2) == fd.ERR_INVALID_ARG
    assert send(pos=None) == fd.ERR_INVALID_ARG
    assert send(k=0) == fd.ERR_INVALID_ARG
    assert send(k=33) == fd.ERR_INVALID_ARG
    assert send(T=-1) == fd.ERR_SHAPE
    assert send(R=1 << 31) == fd.ERR_SHAPE
    assert send(C=24) == fd.ERR_SHAPE
    assert send(rq=None) == fd.ERR_INVALID_ARG
    assert send(q=A) == fd.ERR_INVALID_ARG             # codes without their factors
    assert send(x=A + 8) == fd.ERR_ALIGN
    assert send(pos=A + 2) == fd.ERR_ALIGN
    back = lambda y=A, dt=0, R=20, C=256, pos=A, w=A, T=10, k=2, out=A: L.moe_combine(y, dt, R, C, pos, w, T, k, out, None)  # noqa: E731
    assert back(y=None) == fd.ERR_INVALID_ARG
    assert back(out=None) == fd.ERR_INVALID_ARG
    assert back(dt=2) == fd.ERR_INVALID_ARG
    assert back(C=8) == fd.ERR_SHAPE
    assert back(w=A + 1) == fd.ERR_ALIGN
    assert back(out=A + 4) == fd.ERR_ALIGN
    grad = lambda d=A, y=A, w=A, dy=A, dw=A, k=2: L.moe_combine_bwd(d, y, 1, 20, 256, A, w, 10, k, dy, dw, None)  # noqa: E731
    assert grad(d=None) == fd.ERR_INVALID_ARG
    assert grad(dy=None, dw=None) == fd.ERR_INVALID_ARG
    assert grad(y=None) == fd.ERR_INVALID_ARG          # dweight needs y
    assert grad(w=None) == fd.ERR_INVALID_ARG          # dy needs the weights
    assert grad(k=64) == fd.ERR_INVALID_ARG
    assert grad(dy=A + 8) == fd.ERR_ALIGN


def test_activation_entries_refuse_on_the_host(fd):
    L = fd._lib
    fwd = lambda h=A, dt=1, act=3, R=40, C=144, off=None, g=0, fmt=0, gq=A, gs=A, hq=A, hs=A: L.fp8_block_act(  # noqa: E731
        h, dt, act, R, C, off, g, fmt, gq, gs, hq, hs, None)
    assert fwd(h=None) == fd.ERR_INVALID_ARG
    assert fwd(dt=2) == fd.ERR_INVALID_ARG
    assert fwd(act=4) == fd.ERR_INVALID_ARG
    assert fwd(act=-1) == fd.ERR_INVALID_ARG
    assert fwd(fmt=2) == fd.ERR_INVALID_ARG
    assert fwd(R=-1) == fd.ERR_SHAPE
    assert fwd(C=136) == fd.ERR_SHAPE
    assert fwd(g=2) == fd.ERR_INVALID_ARG
    assert fwd(off=A + 2, g=2) == fd.ERR_ALIGN
    assert fwd(gq=None) == fd.ERR_INVALID_ARG
    assert fwd(hs=None) == fd.ERR_INVALID_ARG
    assert fwd(h=A + 8) == fd.ERR_ALIGN
    ws = fd.fp8_cast_workspace_size(40, 288)
    bwd = lambda dg=A, dt=1, act=3, R=40, C=144, hq=A, hf=0, off=None, g=0, fmt=1, dq=A, ds=A, dt_=A, st=A, gq=A, gs=A, db=None, w=None, wb=0: (  # noqa: E731
        L.fp8_block_dact(dg, dt, act, R, C, hq, hf, A, off, g, fmt, dq, ds, dt_, st, gq, gs, db, w, wb, None))
    assert bwd(dg=None) == fd.ERR_INVALID_ARG
    assert bwd(hq=None) == fd.ERR_INVALID_ARG
    assert bwd(hf=2) == fd.ERR_INVALID_ARG
    assert bwd(fmt=-1) == fd.ERR_INVALID_ARG
    assert bwd(act=7) == fd.ERR_INVALID_ARG
    assert bwd(C=24) == fd.ERR_SHAPE
    assert bwd(dq=None, ds=None, dt_=None, st=None, gq=None, gs=None) == fd.ERR_INVALID_ARG
    assert bwd(ds=None) == fd.ERR_INVALID_ARG
    assert bwd(gq=None) == fd.ERR_INVALID_ARG
    assert bwd(off=A, g=4, db=A, w=A, wb=1 << 20) == fd.ERR_INVALID_ARG  # no bias gradient per group
    assert bwd(db=A) == fd.ERR_WORKSPACE
    assert bwd(db=A, w=A, wb=ws - 1) == fd.ERR_WORKSPACE                # of both halves' columns
    assert bwd(db=A, w=A + 8, wb=ws) == fd.ERR_ALIGN
    assert bwd(gq=A + 8) == fd.ERR_ALIGN
    rec = lambda q=A, f=0, S=40, R=40, C=144, ix=None, off=None, g=0, fmt=0, cq=A, cs=A: L.fp8_block_recode(  # noqa: E731
        q, f, A, S, R, C, ix, off, g, fmt, cq, cs, None)
    assert rec(q=None) == fd.ERR_INVALID_ARG
    assert rec(f=2) == fd.ERR_INVALID_ARG
    assert rec(fmt=2) == fd.ERR_INVALID_ARG
    assert rec(R=41) == fd.ERR_SHAPE                   # more rows than there are, without an index
    assert rec(S=-1) == fd.ERR_SHAPE
    assert rec(C=40) == fd.ERR_SHAPE
    assert rec(cs=None) == fd.ERR_INVALID_ARG
    assert rec(ix=A + 2) == fd.ERR_ALIGN
    assert rec(off=A, g=1025) == fd.ERR_INVALID_ARG
    assert fd.fp8dl_last_error() != ""


def test_binding_refuses_shapes_types_strides_and_cpu_tensors(fd):
    i32, f32, u8 = (lambda *s, d=d: torch.zeros(s, dtype=d) for d in (torch.int32, torch.float32, torch.uint8))
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    T, E, k = 6, 10, 3
    good = dict(expert=i32(T, k), weight=f32(T, k), position=i32(T, k), token=i32(T * k), offsets=i32(E + 1), counts=i32(E),
                slope=f32(E), loss=f32(1), workspace=u8(4096))
    for kw in (dict(expert=i32(T, k).long()), dict(weight=f32(k, T)), dict(token=i32(T)), dict(offsets=i32(E)), dict(loss=f32(2)),
               dict(position=i32(k, T).t()), dict(valid=f32(T)), dict(valid=torch.ones(T + 1, dtype=torch.bool)), {}):
        with pytest.raises(ValueError):  # the last one is well-formed, but on the CPU
            fd.moe_route(bf(T, E), **dict(good, **kw))
    with pytest.raises(TypeError):
        fd.moe_route(bf(T, E).half(), **good)
    with pytest.raises(ValueError):
        fd.moe_route(bf(E, T).t(), **good)
    with pytest.raises(ValueError):
        fd.moe_route_bwd(bf(T, E), i32(T, k), f32(T, k), f32(T, E))  # dlogits of another type
    for kw in (dict(row_s=f32(2, 12)), dict(q=u8(5, 256), s=f32(2, 6)), dict(position=i32(5, 2)), {}):
        with pytest.raises(ValueError):
            fd.fp8_block_dispatch(bf(6, 256), 0, **dict(dict(position=i32(6, 2), row_q=u8(13, 256), row_s=f32(2, 13)), **kw))
    with pytest.raises(ValueError):
        fd.moe_combine(bf(12, 256), i32(6, 2), f32(6, 256))          # out of another type
    with pytest.raises(ValueError):
        fd.moe_combine(bf(12, 256), i32(6, 2), bf(6, 256), weight=f32(6, 3))
    with pytest.raises(ValueError):
        fd.moe_combine_bwd(bf(6, 256), bf(12, 256), i32(6, 2), f32(6, 2))
    with pytest.raises(ValueError):
        fd.moe_combine_bwd(bf(6, 256), bf(11, 256), i32(6, 2), f32(6, 2), dy=bf(12, 256), dweight=f32(6, 2))
    with pytest.raises(ValueError):                                   # a gated activation's h has both halves
        fd.fp8_block_act(bf(5, 144), fd.ACT_SWIGLU, 0, u8(5, 144), f32(2, 5))
    with pytest.raises(ValueError):
        fd.fp8_block_act(bf(5, 288), fd.ACT_SWIGLU, 0, u8(5, 144), f32(2, 5), h_q=u8(5, 288), h_s=f32(2, 5))
    with pytest.raises(ValueError):
        fd.fp8_block_dact(bf(5, 144), u8(5, 288), 0, f32(3, 5), fd.ACT_SWIGLU, 0, dh_qt=u8(288, 128), dh_st=f32(1, 144))
    with pytest.raises(ValueError):
        fd.fp8_block_recode(u8(5, 144), 0, f32(2, 5), 0, u8(144, 128), f32(1, 144), offsets=i32(1))
    with pytest.raises(ValueError):
        fd.fp8_block_recode(u8(5, 144), 0, f32(2, 5), 0, u8(144, 128), f32(1, 144))  # on the CPU


def test_reference_routing_by_hand():
    l = np.log(np.array([[4.0, 2.0, 1.0, 1.0], [1.0, 1.0, 1.0, 1.0], [1.0, 2.0, 4.0, 1.0]]))
    l[2, 0] = -np.inf
    r = mr.route(l, 2, valid=[1, 0, 1])
    assert r["expert"].tolist() == [[0, 1], [-1, -1], [2, 1]]
    assert np.allclose(r["weight"], [[2 / 3, 1 / 3], [0, 0], [2 / 3, 1 / 3]])
    assert r["counts"].tolist() == [1, 2, 1, 0] and r["offsets"].tolist() == [0, 1, 3, 4, 4]
    assert r["position"].tolist() == [[0, 1], [-1, -1], [3, 2]] and r["token"].tolist() == [0, 0, 2, 2, -1, -1]
    P = np.array([4 / 8, 2 / 8 + 2 / 7, 1 / 8 + 4 / 7, 1 / 8 + 1 / 7]) / 2
    assert np.isclose(r["loss"], 4 * (np.array([1, 2, 1, 0]) / 4 * P).sum())
    even = mr.route(np.zeros((8, 4)) + np.eye(4)[np.arange(8) % 4] * 1e-9, 1)
    assert np.isclose(even["loss"], 1.0)  # even counts and probabilities


@pytest.mark.parametrize("normalize", [False, True])
def test_reference_gradient_by_differences(normalize):
    rng = np.random.default_rng(7)
    l, G, dl = rng.standard_normal((5, 6)), rng.standard_normal((5, 2)), 0.3
    r = mr.route(l, 2, normalize=normalize)
    d, _ = mr.route_grad(r, G, dl, normalize)
    f = lambda x: (lambda q: (q["weight"] * G).sum() + dl * q["loss"])(mr.route(x, 2, normalize=normalize))  # noqa: E731
    for i in np.ndindex(l.shape):
        v = np.zeros_like(l)
        v[i] = 1e-6
        assert abs((f(l + v) - f(l - v)) / 2e-6 - d[i]) < 1e-7


@pytest.mark.parametrize("kind", range(4))
def test_reference_activation_derivative_by_differences(kind):
    a = np.linspace(-6, 6, 49)
    d = (mr.act(a + 1e-6, kind)[0] - mr.act(a - 1e-6, kind)[0]) / 2e-6
    assert np.max(np.abs(d - mr.act(a, kind)[1])) < 1e-8
