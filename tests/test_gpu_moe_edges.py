"""Expert routing, token exchange and activations kept in 8 bits where their arithmetic or their indices reach an end."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_reference as br
import moe_reference as mr
import test_gpu_route
import workloads as wl
from conftest import ROOT
from helpers import gpu
from test_gpu_route import Buffers, check, host

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


def test_tokens_of_many_experts_over_many_tiles():
    """1024 experts, 32 choices, several tokens a lane group in every CTA, a ragged end; most of the tokens want the same
    few experts."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    T, E, k = 6001, 1024, 32
    l = wl.normal((T, E), 1.0, wl.generator(431, "many"), torch.float32)
    l[:, 500:540] += 4.0
    for dtype in (torch.bfloat16, torch.float32):
        x = l.to(dtype)
        r = mr.route(x.double().numpy(), k)
        b = Buffers(fd, T, E, k, dev)
        b.run(fd, x.to(dev))
        check(b, x.double().numpy(), r)


def test_factors_of_maxima_of_every_size():
    """A block each for 2^18 maxima: random bit patterns (subnormal ones too), and all that lie around the floor of the
    maximum and the end of the range."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    N, C = 1 << 18, 16
    bits = torch.randint(0, 0x7f800000, (N,), generator=wl.generator(432, "bits")).int()
    around = torch.cat([torch.arange(-500, 500) + b for b in (0x00800000, 0x0d800000, 0x3f800000, 0x43e00000, 0x47600000)] +
                       [torch.arange(0x7f7ffc00, 0x7f800000), torch.arange(0, 500)]).int()
    bits[:around.numel()] = around
    x = torch.zeros((N, C))
    x[torch.arange(N), torch.arange(N) % C] = bits.view(torch.float32)
    pos = torch.arange(N, dtype=torch.int32, device=dev)[:, None].contiguous()
    for fmt in (0, 1):
        q, s = torch.empty((N, C), dtype=torch.uint8, device=dev), torch.empty((1, N), device=dev)
        fd.fp8_block_dispatch(x.to(dev), fmt, pos, q, s)
        want_q, want_s = br.rows(x.numpy(), fmt)
        assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(q.cpu().numpy(), want_q)


OFFSETS = [[50, 10, 400, -7, 90, (1 << 31) - 1], [0, 300, 0, 300, 0, 300], [300, 0], [-(1 << 31), 5, 5, 290], [7, 7, 7]]


@pytest.mark.parametrize("off", OFFSETS)
def test_offsets_out_of_order(off):
    """Offsets that go back, overlap or leave the matrix: what fp8_block_quantize makes of them, nothing outside."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    R, C, G = 300, 272, len(off) - 1
    T, guard = fd.fp8_block_padded_rows(R, G), 4096
    o = torch.tensor(off, dtype=torch.int32, device=dev)
    u8, f32 = (lambda n: torch.full((n + 2 * guard,), 0xAB, dtype=torch.uint8, device=dev)), (lambda n: torch.full((n + 2 * guard,), -7.0, device=dev))
    every = []

    def buffer(make, *shape):
        n = int(np.prod(shape))
        every.append(make(n))
        return every[-1][guard:guard + n].view(shape)

    x = wl.normal((R, C), 1.0, wl.generator(433, "x"), torch.float32)
    q, s = br.rows(x.numpy(), 0)
    v = torch.from_numpy(q).view(torch.float8_e4m3fn).float() * torch.from_numpy(s).t().repeat_interleave(128, 1)[:, :C]
    cq, cs, wq, ws = buffer(u8, C, T), buffer(f32, T // 128, C), buffer(u8, C, T), buffer(f32, T // 128, C)
    fd.fp8_block_quantize(v.to(dev), fd.E4M3, col_q=wq, col_s=ws, offsets=o)
    fd.fp8_block_recode(torch.from_numpy(q).to(dev), 0, torch.from_numpy(s).to(dev), 0, cq, cs, offsets=o)
    assert torch.equal(cq, wq) and torch.equal(cs, ws)
    h = wl.normal((R, 2 * C), 1.0, wl.generator(433, "h"), torch.bfloat16).to(dev)
    dg = wl.normal((R, C), 1.0, wl.generator(433, "dg"), torch.bfloat16).to(dev)
    gq, gs, hq, hs = buffer(u8, R, C), buffer(f32, 3, R), buffer(u8, R, 2 * C), buffer(f32, 5, R)
    fd.fp8_block_act(h, fd.ACT_SWIGLU, 0, gq, gs, h_q=hq, h_s=hs, offsets=o)
    fd.fp8_block_act(h, fd.ACT_SWIGLU, 0, gq, gs, h_q=hq, h_s=hs)
    dq, ds, dt, dts, gt, gts = (buffer(u8, R, 2 * C), buffer(f32, 5, R), buffer(u8, 2 * C, T), buffer(f32, T // 128, 2 * C), buffer(u8, C, T),
                                buffer(f32, T // 128, C))
    fd.fp8_block_dact(dg, hq, 0, hs, fd.ACT_SWIGLU, 0, dh_q=dq, dh_s=ds, dh_qt=dt, dh_st=dts, g_qt=gt, g_st=gts, offsets=o)
    torch.cuda.synchronize()
    for t in every:
        value = 0xAB if t.dtype is torch.uint8 else -7.0
        assert torch.all(t[:guard] == value) and torch.all(t[-guard:] == value)


def test_as_many_groups_as_there_can_be():
    """1024 groups, most of them empty or short: the transposed codes of each group are those of a call for it alone, the
    codes along the rows those of a call without groups."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    R, C, G = 3001, 272, 1024
    length = torch.randint(0, 6, (G,), generator=wl.generator(434, "n"))
    length[::3] = 0
    length[700] = 500
    off = torch.cat([torch.zeros(1, dtype=torch.long), length.cumsum(0)])
    assert off[-1] <= R
    o, T, n = off.int().to(dev), fd.fp8_block_padded_rows(R, G), int(off[-1])
    h = wl.normal((R, 2 * C), 1.0, wl.generator(434, "h"), torch.bfloat16).to(dev)
    dg = wl.normal((R, C), 1.0, wl.generator(434, "dg"), torch.bfloat16).to(dev)
    u8, f32 = (lambda *s: torch.full(s, 0xAB, dtype=torch.uint8, device=dev)), (lambda *s: torch.full(s, -7.0, device=dev))
    gq, gs, hq, hs = u8(R, C), f32(3, R), u8(R, 2 * C), f32(5, R)
    fd.fp8_block_act(h, fd.ACT_SWIGLU, 0, gq, gs, h_q=hq, h_s=hs)

    def back(lo, hi, offsets=None, T=None):
        m = hi - lo
        T = (m + 127) // 128 * 128 if T is None else T
        b = dict(dh_q=u8(m, 2 * C), dh_s=f32(5, m), dh_qt=u8(2 * C, T), dh_st=f32(T // 128, 2 * C), g_qt=u8(C, T), g_st=f32(T // 128, C))
        fd.fp8_block_dact(dg[lo:hi], hq[lo:hi], 0, hs[:, lo:hi].contiguous(), fd.ACT_SWIGLU, 0, offsets=offsets, **b)
        cq, cs = u8(2 * C, T), f32(T // 128, 2 * C)
        fd.fp8_block_recode(hq[lo:hi], 0, hs[:, lo:hi].contiguous(), 1, cq, cs, offsets=offsets)
        return dict(b, cq=cq, cs=cs)

    got, whole = back(0, R, o, T), back(0, R)
    assert torch.equal(got["dh_q"][:n], whole["dh_q"][:n]) and torch.equal(got["dh_s"][:, :n], whole["dh_s"][:, :n])
    assert torch.all(got["dh_q"][n:] == 0xAB) and torch.all(got["dh_s"][:, n:] == -7)
    at = 0
    for g in range(G):
        lo, hi = int(off[g]), int(off[g + 1])
        blocks = (hi - lo + 127) // 128
        if hi > lo and (g % 50 == 1 or g == 700):
            alone = back(lo, hi)
            for name in ("dh_qt", "g_qt", "cq"):
                assert torch.equal(got[name][:, 128 * at:128 * (at + blocks)], alone[name]), (name, g)
            for name in ("dh_st", "g_st", "cs"):
                assert torch.equal(got[name][at:at + blocks], alone[name]), (name, g)
        at += blocks
    assert torch.all(got["cq"][:, 128 * at:] == 0xAB) and torch.all(got["dh_qt"][:, 128 * at:] == 0xAB)


def test_recode_without_source_rows():
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    C, R = 144, 200
    index = torch.arange(R, dtype=torch.int32, device=dev)
    q, s = torch.empty((0, C), dtype=torch.uint8, device=dev), torch.empty((2, 0), device=dev)
    cq, cs = torch.full((C, 256), 0xAB, dtype=torch.uint8, device=dev), torch.zeros((2, C), device=dev)
    fd.fp8_block_recode(q, 0, s, 0, cq, cs, index=index)
    assert torch.all(cq == 0) and torch.all(cs == 1)


def test_two_graphs_that_share_a_workspace():
    """Captured routing calls of different sizes over one workspace, replayed in turn with new logits."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    shapes = [(9000, 40, 4), (3001, 300, 8), (20, 64, 6)]
    ws = torch.empty(max(fd.moe_route_workspace_size(T, E) for T, E, _ in shapes), dtype=torch.uint8, device=dev)
    out = [(Buffers(fd, T, E, k, dev, ws=ws), torch.zeros((T, E), dtype=torch.bfloat16, device=dev)) for T, E, k in shapes]
    side = torch.cuda.Stream()
    graphs = []
    for b, l in out:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            b.run(fd, l)
        graphs.append(g)
    for turn in range(3):
        logits = [wl.normal((T, E), 2.0, wl.generator(435, "%d,%d" % (turn, T)), torch.bfloat16) for T, E, _ in shapes]
        for (b, l), x, g in zip(out, logits, graphs):
            l.copy_(x)
            g.replay()
        torch.cuda.synchronize()
        for (b, _), x, (T, E, k) in zip(out, logits, shapes):
            b.token[int(b.offsets[-1]):] = -7
            check(b, x.double().numpy(), mr.route(x.double().numpy(), k))


SCRIPT = r'''
import threading, torch
import fp8_delayed_scaling_gb300 as fd
dev = torch.device("cuda", 0)
torch.cuda.set_device(dev)
N, T, E, k, C, G = 8, 700, 1000, 4, 272, 5
g = torch.Generator().manual_seed(9)
logits = [torch.randn(T, E, generator=g).to(dev) for _ in range(N)]
hs = [torch.randn(T, 2 * C, generator=g).bfloat16().to(dev) for _ in range(N)]
dgs = [torch.randn(T, C, generator=g).bfloat16().to(dev) for _ in range(N)]
off = torch.tensor([0, 100, 100, 350, 600, 699], dtype=torch.int32, device=dev)
P = fd.fp8_block_padded_rows(T, G)

def work(i, out):
    torch.cuda.set_device(dev)
    with torch.cuda.stream(torch.cuda.Stream()):
        u8, f32 = (lambda *s: torch.zeros(s, dtype=torch.uint8, device=dev)), (lambda *s: torch.zeros(s, device=dev))
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
        e, w, p, t, o = i32(T, k), f32(T, k), i32(T, k), i32(T * k), i32(E + 1)
        fd.moe_route(logits[i], e, w, p, t, o, workspace=u8(fd.moe_route_workspace_size(T, E)))
        gq, gs, hq, hss = u8(T, C), f32(3, T), u8(T, 2 * C), f32(5, T)
        fd.fp8_block_act(hs[i], fd.ACT_SWIGLU, fd.E4M3, gq, gs, h_q=hq, h_s=hss, offsets=off)
        dq, ds, dt, dts, gt, gts = u8(T, 2 * C), f32(5, T), u8(2 * C, P), f32(P // 128, 2 * C), u8(C, P), f32(P // 128, C)
        fd.fp8_block_dact(dgs[i], hq, fd.E4M3, hss, fd.ACT_SWIGLU, fd.E4M3, dh_q=dq, dh_s=ds, dh_qt=dt, dh_st=dts, g_qt=gt, g_st=gts, offsets=off)
        cq, cs = u8(2 * C, P), f32(P // 128, 2 * C)
        fd.fp8_block_recode(hq, fd.E4M3, hss, fd.E4M3, cq, cs, offsets=off)
        rq, rs = u8(T * k, C), f32(3, T * k)
        fd.fp8_block_dispatch(dgs[i], fd.E4M3, p, rq, rs)
        y = torch.empty_like(dgs[i])
        fd.moe_combine(dgs[i].repeat(k, 1), p, y, weight=w)
        torch.cuda.current_stream().synchronize()
        out[i] = [x.cpu() for x in (e, w, p, t, o, gq, gs, hq, hss, dq, ds, dt, dts, gt, gts, cq, cs, rq, rs, y)]

first, again = [None] * N, [None] * N
torch.cuda.synchronize()
barrier = threading.Barrier(N)
def run(i):
    barrier.wait()
    work(i, first)
ts = [threading.Thread(target=run, args=(i,)) for i in range(N)]
for t in ts: t.start()
for t in ts: t.join()
for i in range(N):
    work(i, again)
    assert first[i] is not None, i
    assert all(torch.equal(a, b) for a, b in zip(first[i], again[i])), i
print("threads ok")
'''


def test_first_calls_from_several_threads_and_streams():
    env = dict(os.environ)
    env["PYTHONPATH"] = ROOT + os.pathsep + env.get("PYTHONPATH", "")
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "threads ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]


@pytest.mark.parametrize("E", [1, 6, 16, 24, 50, 64, 100, 200, 256, 400, 1024])
def test_choices_among_all_bf16_values(E):
    """Every bit pattern of bf16, subnormal ones, both zeros, infinities and NaN among them: the choices are those of the
    values' order, equal ones by the lower expert."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    k = min(E, 16)
    T = max(200, 65536 // E + 1)
    n = T * E
    bits = torch.randperm(n, generator=wl.generator(436, "p%d" % E)) % 65536
    bits[::5] = torch.tensor([0, 0x8000, 1, 0x8001, 0xff80, 0x7f80, 0x7fc0, 0xffc0])[torch.arange(bits[::5].numel()) % 8]
    l = (bits - 65536 * (bits >= 32768)).to(torch.int16).view(torch.bfloat16).view(T, E)
    with np.errstate(invalid="ignore"):
        r = mr.route(l.double().numpy(), k)
    b = Buffers(fd, T, E, k, dev)
    b.run(fd, l.to(dev))
    for name in ("expert", "position", "offsets", "counts"):
        assert np.array_equal(getattr(b, name).cpu().numpy(), r[name]), name
    nan = np.isnan(l.double().numpy()).any(1) | (l.double().numpy() == np.inf).any(1)
    assert np.array_equal(np.isnan(host(b.weight))[:, 0], nan & r["has"][:, 0])


@pytest.mark.parametrize("act", [0, 2])
def test_gelu_of_blocks_that_hold_small_results_only(act):
    """Blocks of one value each from -13 to 13: their factors are the results, to a relative error.  In units of 2^-24:
    the exponent's two roundings and its constant (3 of a^2 / 2), 2^x (4), the ratio (9 and 1/x: 3), products (4) and
    the factor (4).  The derivative's difference of ratio and phi(0) x is at most 2.2 times smaller than their sum
    beyond |a| = 1.5."""
    import math

    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    R, C = 2601, 16
    a = torch.linspace(-13, 13, R)
    q, s = torch.full((R, C), 0x38, dtype=torch.uint8), a.abs().view(1, R)  # the code of 1, -1 where a < 0
    q[a < 0] = 0xb8
    gated = act == 2
    hq = torch.cat([q, torch.full((R, C), 0x38, dtype=torch.uint8)], 1) if gated else q
    hs = s  # 2 C columns are one block: u = |a| too
    W = hq.shape[1]
    groups = 1024
    v = a.double().numpy()
    u = np.abs(v) if gated else np.ones(R)
    e = np.exp(-v * v / 2)
    cdf = np.array([0.5 * math.erfc(-x / math.sqrt(2)) for x in v])
    y, d = v * cdf * u, (cdf + v * e / math.sqrt(2 * math.pi)) * u
    tol = (1.5 * v * v + 30) * mr.EPS
    h = (torch.cat([a[:, None].expand(R, C), a.abs()[:, None].expand(R, C)], 1) if gated else a[:, None].expand(R, C)).contiguous()
    gq, gs = torch.zeros((R, C), dtype=torch.uint8, device=dev), torch.zeros((1, R), device=dev)
    fd.fp8_block_act(h.to(dev), act, 0, gq, gs)
    small = np.abs(y) > 2.0 ** -99  # a block's scale is that of a maximum of 2^-100 at least: below it the factor says nothing
    got = host(gs)[0] * 448
    assert np.all((np.abs(got - np.abs(y)) <= tol * np.abs(y))[small & (v != 0)])
    # backward: groups of one row, so that a column's block holds one value
    for lo in range(0, R, groups):
        n = min(groups, R - lo)
        off = torch.arange(n + 1, dtype=torch.int32, device=dev)
        T = fd.fp8_block_padded_rows(n, n)
        gt, gts = torch.zeros((C, T), dtype=torch.uint8, device=dev), torch.zeros((T // 128, C), device=dev)
        dt, dts = torch.zeros((W, T), dtype=torch.uint8, device=dev), torch.zeros((T // 128, W), device=dev)
        fd.fp8_block_dact(torch.ones((n, C), device=dev), hq[lo:lo + n].contiguous().to(dev), 0, hs[:, lo:lo + n].contiguous().to(dev), act, 0,
                          dh_qt=dt, dh_st=dts, g_qt=gt, g_st=gts, offsets=off)
        at = slice(lo, lo + n)
        w = small[at] & (v[at] != 0)
        assert np.all((np.abs(host(gts)[:n, 0] * 448 - np.abs(y[at])) <= tol[at] * np.abs(y[at]))[w])
        far = w & (np.abs(v[at]) > 1.5) & (np.abs(d[at]) > 2.0 ** -99)
        assert np.all((np.abs(host(dts)[:n, 0] * 448 - np.abs(d[at])) <= 2.2 * tol[at] * np.abs(d[at]))[far])


@pytest.mark.parametrize("T,E,k", [(40, 20, 12), (33, 30, 9), (65, 50, 10), (50, 64, 16), (70, 128, 16), (70, 127, 17), (5000, 60, 9)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_more_choices_than_a_quarter_of_a_warp_has_lanes(T, E, k, dtype):
    test_gpu_route.test_route_and_gradient(T, E, k, dtype)


@pytest.mark.parametrize("T,k,C", [(3000, 1, 144), (3000, 2, 272), (2600, 4, 144), (2600, 5, 272), (1300, 8, 528), (1300, 9, 144),
                                   (11001, 1, 144), (5200, 2, 528)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_exchange_of_many_tokens(T, k, C, dtype):
    """One warp a token in the gradient; sums of k products in order, C products over a lane, a tree and a few warps."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    g = wl.generator(437, "x%d,%d" % (T, k))
    R = T * k + 7
    pos = torch.randperm(R, generator=g)[:T * k].view(T, k).int()
    pos[torch.rand((T, k), generator=g) < 0.1] = -1
    y, x = wl.normal((R, C), 1.0, g, dtype), wl.normal((T, C), 1.0, g, dtype)
    w = torch.rand((T, k), generator=g) + 0.1
    yd, xd, pd, wd = y.to(dev), x.to(dev), pos.to(dev), w.to(dev)
    out, dy, dw = torch.empty_like(xd), torch.full_like(yd, 9.0), torch.empty_like(wd)
    fd.moe_combine(yd, pd, out, weight=wd)
    fd.moe_combine_bwd(xd, yd, pd, wd, dy=dy, dweight=dw)
    used = (pos >= 0).numpy()
    rows = np.where(used, pos.numpy(), 0)
    yv, xv, wv = y.double().numpy(), x.double().numpy(), np.where(used, w.double().numpy(), 0.0)
    terms = wv[:, :, None] * yv[rows]
    half = torch.finfo(dtype).eps / 2
    want, size = terms.sum(1), np.abs(terms).sum(1)
    assert np.all(np.abs(host(out) - want) <= half * np.abs(want) * 1.01 + (k + 1) * mr.EPS * size)
    want_dy = np.full((R, C), 9.0)
    want_dy[rows[used]] = (wv[:, :, None] * xv[:, None, :])[used]
    assert np.all(np.abs(host(dy) - want_dy) <= half * np.abs(want_dy) * 1.01 + mr.EPS * np.abs(want_dy))
    prod = xv[:, None, :] * yv[rows]
    want_dw, size_dw = np.where(used, prod.sum(2), 0.0), np.abs(prod).sum(2)
    assert np.all(np.abs(host(dw) - want_dw) <= (C / 32 + 16) * mr.EPS * size_dw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", range(4))
def test_more_jobs_than_there_are_threads_blocks(act, dtype):
    """Thread blocks that walk several jobs and tiles, with halves of h that do not start on a block: rows, tiles and their
    sums are, bit by bit, those of calls for 128 rows, and dbias the sum of theirs."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    R, C = 3000, 1040
    W = 2 * C if act >= 2 else C
    B, D = (C + 127) // 128, (W + 127) // 128
    g = wl.generator(438, "h%d" % act)
    h, dg = wl.normal((R, W), 1.5, g, dtype).to(dev), wl.normal((R, C), 1.0, g, dtype).to(dev)

    def run(h, dg):
        n = h.shape[0]
        T = (n + 127) // 128 * 128
        u8, f32 = (lambda *s: torch.full(s, 0xAB, dtype=torch.uint8, device=dev)), (lambda *s: torch.full(s, -7.0, device=dev))
        b = dict(gq=u8(n, C), gs=f32(B, n), hq=u8(n, W), hs=f32(D, n), dq=u8(n, W), ds=f32(D, n), dt=u8(W, T), dts=f32(T // 128, W),
                 gt=u8(C, T), gts=f32(T // 128, C), db=f32(W))
        only = u8(n, C), f32(B, n)
        fd.fp8_block_act(h, act, 0, *only)
        fd.fp8_block_act(h, act, 0, b["gq"], b["gs"], h_q=b["hq"], h_s=b["hs"])
        assert torch.equal(only[0], b["gq"]) and torch.equal(only[1], b["gs"])
        ws = torch.empty(fd.fp8_cast_workspace_size(n, W), dtype=torch.uint8, device=dev)
        fd.fp8_block_dact(dg, b["hq"], 0, b["hs"], act, 1, dh_q=b["dq"], dh_s=b["ds"], dh_qt=b["dt"], dh_st=b["dts"], g_qt=b["gt"],
                          g_st=b["gts"], dbias=b["db"], workspace=ws)
        return b

    whole = run(h, dg)
    total, size = torch.zeros(W, dtype=torch.float64, device=dev), torch.zeros(W, dtype=torch.float64, device=dev)
    for lo in range(0, R, 128):
        hi = min(lo + 128, R)
        part = run(h[lo:hi], dg[lo:hi])
        for name in ("gq", "hq", "dq"):
            assert torch.equal(whole[name][lo:hi], part[name]), (name, lo)
        for name in ("gs", "hs", "ds"):
            assert torch.equal(whole[name][:, lo:hi], part[name]), (name, lo)
        for name in ("dt", "gt"):
            assert torch.equal(whole[name][:, lo:lo + 128], part[name]), (name, lo)
        for name in ("dts", "gts"):
            assert torch.equal(whole[name][lo // 128:lo // 128 + 1], part[name]), (name, lo)
        total += part["db"].double()
        size += part["db"].double().abs()
    assert torch.all((whole["db"].double() - total).abs() <= (R // 128 + 2) * mr.EPS * size)
