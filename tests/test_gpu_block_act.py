"""fp8_block_act, fp8_block_dact and fp8_block_recode.  The checkpoint and transposed codes made from codes: bit by bit.
Computed values: each code stands for the 64-bit value within half a step of the format, the block's
rounding and what the fp32 activation may be off by."""
import numpy as np
import pytest
import torch

import block_reference as br
import moe_reference as mr
import workloads as wl
from helpers import gpu

pytestmark = pytest.mark.gpu

EPS = mr.EPS
STEP = {0: (2.0 ** -4, 2.0 ** -10), 1: (2.0 ** -3, 2.0 ** -17)}  # half a step of a value, half the smallest code


def f64(t):
    return t.detach().double().cpu().numpy()


def groups(rows, n, behind, name):
    """Offsets that begin behind a few rows, with empty groups, and leave `behind` rows."""
    g = np.random.default_rng(wl.generator(420, name).initial_seed() % (1 << 32))
    lo = min(2, max(0, rows - behind))
    cuts = np.sort(g.integers(lo, max(lo, rows - behind) + 1, n - 1)) if n > 1 else np.zeros(0, int)
    return np.concatenate([[lo], cuts, [max(lo, rows - behind)]]).astype(np.int64)


def check_codes(q, s, fmt, value, err, axis_blocks, what):
    """q (codes, blocks of 128 along axis 1), s [blocks, rows] against fp64 `value` known to `err`; axis_blocks: the
    first and last + 1 of the 128-blocks' columns."""
    half, sub = STEP[fmt]
    v = torch.from_numpy(np.ascontiguousarray(q)).view(br.F8[fmt]).double().numpy()
    for b, (lo, hi) in enumerate(axis_blocks):
        if hi <= lo:
            continue
        x, e = value[:, lo:hi], err[:, lo:hi]
        amax, emax = np.abs(x).max(1, keepdims=True), e.max(1, keepdims=True)
        f = s[b][:, None].astype(np.float64)
        live = (amax > 2 * emax) & (amax > 2.0 ** -99)
        want = amax / br.MAX[fmt]
        assert np.all((np.abs(f - want) <= emax / br.MAX[fmt] + 4 * EPS * want)[live]), what + ": factors"
        # scale, its reciprocal, the scaled value: a few roundings of fp32 beside the code's own
        bound = (half * np.abs(x) + sub * (amax + emax) / br.MAX[fmt]) * (1 + 2.0 ** -18) + 2.0 ** -21 * np.abs(x) + 2 * e + 2.0 ** -100
        bad = ~(np.abs(v[:, lo:hi] * f - x) <= bound)
        assert not bad.any(), "%s: %d of %d codes of block %d off" % (what, bad.sum(), bad.size, b)


def along(n):
    return [(c, min(c + 128, n)) for c in range(0, n, 128)]


def padded(x, off, T):
    """x's rows by group, each padded to a multiple of 128 with zeros; and the blocks' columns."""
    out, at, spans = np.zeros((x.shape[1], T)), 0, []
    for lo, hi in zip(off[:-1], off[1:]):
        for r in range(lo, hi, 128):
            n = min(r + 128, hi) - r
            out[:, at:at + n] = x[r:r + n].T
            spans.append((at, at + n))
            at += 128
    return out, spans


def wide(act, C):
    return 2 * C if act >= 2 else C


SHAPES = [(1, 16, 0, 0), (1, 1408, 3, 0), (2, 144, 0, 0), (5, 128, 2, 1), (127, 112, 0, 0), (128, 256, 1, 0), (129, 272, 0, 0), (300, 400, 7, 20),
          (515, 640, 40, 3), (131, 1040, 0, 0)]


@pytest.mark.parametrize("R,C,G,behind", SHAPES)
@pytest.mark.parametrize("act", range(4))
def test_forward(R, C, G, behind, act):
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    dtype, fmt = ((torch.bfloat16, 0), (torch.float32, 0), (torch.float32, 1))[(R + act) % 3]
    W = wide(act, C)
    h = wl.student_t3((R, W), 1.0, wl.generator(421, "h%d,%d" % (R, C)), dtype)
    if R > 4:
        h[3] = 0.0
    off = groups(R, G, behind, "f%d" % R) if G else None
    o = None if off is None else torch.from_numpy(off).int().to(dev)
    lo, hi = (0, R) if off is None else (int(off[0]), int(off[-1]))
    H = f64(h)
    y, _, ey, _ = mr.act(H[:, :C], act)
    if act >= 2:
        y, ey = y * H[:, C:], ey * np.abs(H[:, C:]) + EPS * np.abs(y * H[:, C:])
    for keep in (True, False):
        gq, gs = torch.full((R, C), 0xAB, dtype=torch.uint8, device=dev), torch.full((br.blocks(C), R), -7.0, device=dev)
        hq, hs = torch.full((R, W), 0xAB, dtype=torch.uint8, device=dev), torch.full((br.blocks(W), R), -7.0, device=dev)
        fd.fp8_block_act(h.to(dev), act, fmt, gq, gs, h_q=hq if keep else None, h_s=hs if keep else None, offsets=o)
        q, s = gq.cpu().numpy(), gs.cpu().numpy()
        if hi > lo:
            check_codes(q[lo:hi], s[:, lo:hi], fmt, y[lo:hi], ey[lo:hi], along(C), "g")
        for t in (q[:lo], q[hi:], hq.cpu().numpy()[:lo], hq.cpu().numpy()[hi:]):
            assert np.all(t == 0xAB)
        for t in (s[:, :lo], s[:, hi:], hs.cpu().numpy()[:, :lo], hs.cpu().numpy()[:, hi:]):
            assert np.all(t == -7.0)
        if keep:
            want, ws = br.rows(h.float().numpy(), fmt)
            assert np.array_equal(hq.cpu().numpy()[lo:hi], want[lo:hi]) and np.array_equal(hs.cpu().numpy()[:, lo:hi], ws[:, lo:hi])
        else:
            assert torch.all(hq == 0xAB) and torch.all(hs == -7.0)


def _dact(fd, dg, hq, hf, hs, act, fmt, o, dev, parts="rtgb"):
    R, C = dg.shape
    W, G = wide(act, C), 0 if o is None else o.numel() - 1
    T = fd.fp8_block_padded_rows(R, G)
    u8, f32 = (lambda *s: torch.full(s, 0xAB, dtype=torch.uint8, device=dev)), (lambda *s: torch.full(s, -7.0, device=dev))
    b = dict(dh_q=u8(R, W), dh_s=f32(br.blocks(W), R)) if "r" in parts else {}
    if "t" in parts:
        b.update(dh_qt=u8(W, T), dh_st=f32(T // 128, W))
    if "g" in parts:
        b.update(g_qt=u8(C, T), g_st=f32(T // 128, C))
    if "b" in parts and o is None:
        b.update(dbias=f32(W), workspace=torch.empty(fd.fp8_cast_workspace_size(R, W), dtype=torch.uint8, device=dev))
    fd.fp8_block_dact(dg, hq, hf, hs, act, fmt, offsets=o, **b)
    return b


@pytest.mark.parametrize("R,C,G,behind", SHAPES)
@pytest.mark.parametrize("act", range(4))
def test_backward(R, C, G, behind, act):
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    dtype, fmt, hf = ((torch.bfloat16, 0, 0), (torch.float32, 1, 0), (torch.bfloat16, 1, 1))[(R + act) % 3]
    W = wide(act, C)
    h = wl.student_t3((R, W), 1.0, wl.generator(422, "h%d,%d" % (R, C)), torch.bfloat16)
    dg = wl.normal((R, C), 1e-3, wl.generator(422, "g%d,%d" % (R, C)), dtype)
    if R > 4:
        dg[4], h[3] = 0.0, 0.0
    qh, sh = br.rows(h.float().numpy(), hf)
    off = groups(R, G, behind, "b%d" % R) if G else None
    o = None if off is None else torch.from_numpy(off).int().to(dev)
    spans = [0, R] if off is None else off.tolist()
    lo, hi = spans[0], spans[-1]
    T = fd.fp8_block_padded_rows(R, G)
    b = _dact(fd, dg.to(dev), torch.from_numpy(qh).to(dev), hf, torch.from_numpy(sh).to(dev), act, fmt, o, dev)
    code = torch.from_numpy(qh).view(br.F8[hf]).float().numpy()
    H = (code * np.repeat(sh.T, 128, 1)[:, :W]).astype(np.float64)  # fl32(code * factor)
    D = f64(dg)
    y, d, ey, ed = mr.act(H[:, :C], act)
    if act >= 2:
        u = H[:, C:]
        dh, e = np.concatenate([D * u * d, D * y], 1), np.concatenate([np.abs(D * u) * (ed + 3 * EPS * np.abs(d)), np.abs(D) * (ey + EPS * np.abs(y))], 1)
        y, ey = y * u, ey * np.abs(u) + EPS * np.abs(y * u)
    else:
        dh, e = D * d, np.abs(D) * (ed + EPS * np.abs(d))
    q, s = b["dh_q"].cpu().numpy(), b["dh_s"].cpu().numpy()
    if hi > lo:
        check_codes(q[lo:hi], s[:, lo:hi], fmt, dh[lo:hi], e[lo:hi], along(W), "dh")
    assert np.all(q[:lo] == 0xAB) and np.all(q[hi:] == 0xAB) and np.all(s[:, :lo] == -7.0) and np.all(s[:, hi:] == -7.0)
    for name, v, ev, f in (("dh", dh, e, fmt), ("g", y, ey, hf)):
        vt, cols = padded(v, spans, T)
        et, _ = padded(ev, spans, T)
        q, s = b[name + "_qt"].cpu().numpy(), b[name + "_st"].cpu().numpy()
        used = 128 * len(cols)
        check_codes(q, s, f, vt, et, cols, name + " transposed")
        for at, (c0, c1) in enumerate(cols):
            assert np.all(q[:, c1:128 * at + 128] == 0)                   # a group's padding: zero codes
        assert np.all(q[:, used:] == 0xAB) and np.all(s[used // 128:] == -7.0)  # behind the last group
    if o is None:
        assert np.all(np.abs(f64(b["dbias"]) - dh.sum(0)) <= e.sum(0) + R * EPS * (np.abs(dh) + e).sum(0) + 2.0 ** -110)
    # every output alone has the same bits
    for part in "rtgb":
        if part == "b" and o is not None:
            continue
        for k, v in _dact(fd, dg.to(dev), torch.from_numpy(qh).to(dev), hf, torch.from_numpy(sh).to(dev), act, fmt, o, dev, part).items():
            assert k == "workspace" or torch.equal(v, b[k]), (part, k)


@pytest.mark.parametrize("act", range(4))
def test_chain_against_the_unquantised_formula(act):
    """Forward and backward from the same h: dh's codes against the derivative at the kept values, and those against h itself,
    within half a step of the checkpoint."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    R, C = 200, 384
    W = wide(act, C)
    h = wl.normal((R, W), 1.5, wl.generator(423, "h"), torch.bfloat16)
    gq, gs = torch.zeros((R, C), dtype=torch.uint8, device=dev), torch.zeros((3, R), device=dev)
    hq, hs = torch.zeros((R, W), dtype=torch.uint8, device=dev), torch.zeros((W // 128, R), device=dev)
    fd.fp8_block_act(h.to(dev), act, fd.E4M3, gq, gs, h_q=hq, h_s=hs)
    kept = br.values(hq.cpu().numpy(), 0, hs.cpu().numpy(), 1)
    H = f64(h)
    amax = np.abs(H.reshape(R, -1, 128)).max(2).repeat(128, 1)
    assert np.all(np.abs(kept - H) <= (2.0 ** -4 * np.abs(H) + 2.0 ** -10 * amax / 448) * (1 + 2.0 ** -18) + 2.0 ** -21 * np.abs(H))
    ones = torch.ones((R, C), device=dev)
    b = _dact(fd, ones, hq, 0, hs, act, 0, None, dev, "r")
    d = br.values(b["dh_q"].cpu().numpy(), 0, b["dh_s"].cpu().numpy(), 1)
    # central differences of the fp64 activation at the kept values (h^2 f''' / 6 < 1e-8 at h = 1e-4)
    f = lambda x: mr.act(x[:, :C], act)[0] * (x[:, C:] if act >= 2 else 1.0)  # noqa: E731
    h4 = 1e-4
    for half, at in ((0, slice(0, C)),) + (((1, slice(C, W)),) if act >= 2 else ()):
        v = np.zeros_like(kept)
        v[:, at] = h4
        diff = (f(kept + v) - f(kept - v)) / (2 * h4)
        top = np.abs(diff.reshape(R, -1, 128)).max(2).repeat(128, 1)
        assert np.all(np.abs(d[:, at] - diff) <= 2.0 ** -4 * np.abs(diff) * 1.001 + 2.0 ** -10 * top / 448 * 1.001 + 1e-5 * (1 + np.abs(diff)))


@pytest.mark.parametrize("act", range(4))
def test_values_that_are_not_finite(act):
    """Infinities saturate and NaN stays NaN in its own place; the other codes of its blocks are as without them."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    R, C = 140, 272
    W = wide(act, C)
    h = wl.normal((R, W), 1.0, wl.generator(424, "h"), torch.float32)
    clean = h.clone()
    h[5, 7], h[9, 200], h[130, 260] = float("nan"), float("inf"), -float("inf")
    clean[5, 7] = clean[9, 200] = clean[130, 260] = 0.0
    out = []
    for x in (h, clean):
        gq, gs = torch.zeros((R, C), dtype=torch.uint8, device=dev), torch.zeros((3, R), device=dev)
        hq, hs = torch.zeros((R, W), dtype=torch.uint8, device=dev), torch.zeros((br.blocks(W), R), device=dev)
        fd.fp8_block_act(x.to(dev), act, 0, gq, gs, h_q=hq, h_s=hs)
        out.append((gq, gs, hq, hs))
    (gq, gs, hq, hs), (cq, cs, _, _) = out
    want, ws = br.rows(h.numpy(), 0)
    assert np.array_equal(hq.cpu().numpy(), want) and np.array_equal(hs.cpu().numpy(), ws)
    same = torch.ones((R, C), dtype=torch.bool)
    for r, c in ((5, 7), (9, 200), (130, 260)):
        same[r, c] = False
    assert torch.equal(gq.cpu()[same], cq.cpu()[same]) and torch.equal(gs, cs)
    g = gq.cpu().view(torch.float8_e4m3fn).float()
    assert torch.isnan(g[5, 7]) and abs(float(g[9, 200])) == 448
    # backward: a NaN in dg and in the checkpoint
    dg = wl.normal((R, C), 1.0, wl.generator(424, "g"), torch.float32)
    dg[20, 30] = float("nan")
    dg[21, 31] = float("inf")
    b = _dact(fd, dg.to(dev), hq, 0, hs, act, 0, None, dev)
    v = b["dh_q"].cpu().view(torch.float8_e4m3fn).float()
    at = torch.isnan(v).nonzero().tolist()
    want = {(20, 30), (5, 7)} | ({(20, 30 + C), (5, 7 + C)} if act >= 2 else set())
    assert {tuple(x) for x in at} == want
    assert torch.isfinite(b["dh_s"]).all() and torch.isfinite(b["dh_st"]).all() and torch.isfinite(b["g_st"]).all()
    t = b["dh_qt"].cpu().view(torch.float8_e4m3fn).float()[:, :R].t()
    assert torch.equal(torch.isnan(t), torch.isnan(v))


@pytest.mark.parametrize("S,R,C,G,behind,index", [(1, 1, 16, 0, 0, False), (300, 300, 272, 0, 0, False), (300, 129, 272, 0, 0, False),
                                                   (40, 300, 144, 7, 20, True), (515, 515, 640, 40, 3, False), (9, 4, 400, 3, 0, True),
                                                   (700, 1400, 128, 24, 9, True)])
@pytest.mark.parametrize("f,to", [(0, 0), (1, 0), (0, 1), (1, 1)])
def test_recode(S, R, C, G, behind, index, f, to):
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    x = wl.student_t3((S, C), 1.0, wl.generator(425, "x%d" % S), torch.float32)
    if S > 8:
        x[5], x[7, 3], x[8, 9] = 0.0, float("nan"), float("inf")
    q, s = br.rows(x.numpy(), f)
    off = groups(R, G, behind, "r%d" % R) if G else None
    ix = None
    if index:
        ix = torch.randint(0, S, (R,), generator=wl.generator(425, "i")).int()
        ix[::7], ix[3::11] = -1, S  # rows of zeros
        ix[2::13] = -(1 << 31)
    T = fd.fp8_block_padded_rows(R, G)
    cq, cs = torch.full((C, T), 0xAB, dtype=torch.uint8, device=dev), torch.full((T // 128, C), -7.0, device=dev)
    src_q, src_s = (q, s) if index else (q[:R], np.ascontiguousarray(s[:, :R]))
    fd.fp8_block_recode(torch.from_numpy(src_q).to(dev), f, torch.from_numpy(src_s).to(dev), to, cq, cs,
                        offsets=None if off is None else torch.from_numpy(off).int().to(dev), index=None if ix is None else ix.to(dev))
    with np.errstate(invalid="ignore"):
        v = torch.from_numpy(q).view(br.F8[f]).float().numpy() * np.repeat(s.T, 128, 1)[:, :C]
    if index:
        ok = ((ix >= 0) & (ix < S)).numpy()
        v = np.where(ok[:, None], v[np.where(ok, ix.numpy(), 0)], np.float32(0))
    want, ws, used = br.cols(v[:R].astype(np.float32), to, None if off is None else off.tolist())
    got = cq.cpu().numpy()
    nan = torch.from_numpy(want).view(br.F8[to]).float().isnan().numpy()
    assert np.array_equal(got[:, :used][~nan[:, :used]], want[:, :used][~nan[:, :used]])
    assert torch.from_numpy(got).view(br.F8[to]).float().isnan().numpy()[nan].all()
    assert np.array_equal(cs.cpu().numpy()[:used // 128], ws[:used // 128])
    assert np.all(got[:, used:] == 0xAB) and np.all(cs.cpu().numpy()[used // 128:] == -7.0)


def test_no_rows():
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    u8, f32 = (lambda *s: torch.zeros(s, dtype=torch.uint8, device=dev)), (lambda *s: torch.full(s, 7.0, device=dev))
    fd.fp8_block_act(f32(0, 288), fd.ACT_SWIGLU, 0, u8(0, 144), f32(2, 0), h_q=u8(0, 288), h_s=f32(3, 0))
    db = f32(288)
    fd.fp8_block_dact(f32(0, 144), u8(0, 288), 0, f32(3, 0), fd.ACT_SWIGLU, 0, dh_q=u8(0, 288), dh_s=f32(3, 0), dbias=db)
    assert torch.all(db == 0)
    fd.fp8_block_recode(u8(0, 144), 0, f32(2, 0), 0, u8(144, 0), f32(0, 144))
    off = torch.zeros(3, dtype=torch.int32, device=dev)  # rows, but none in a group
    q, s = u8(5, 144), f32(2, 5)
    fd.fp8_block_act(f32(5, 288), fd.ACT_SWIGLU, 0, q, s, offsets=off)
    assert torch.all(q == 0) and torch.all(s == 7)
