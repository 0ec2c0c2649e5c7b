"""Block-scaled FP8 where its arithmetic reaches an end: overlapping groups of more than 2^32 blocks, infinities and NaN in
every place of a block, first calls from several threads, and expert layers element by element."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_reference as br
import workloads as wl
from conftest import ROOT
from helpers import gpu

pytestmark = pytest.mark.gpu


def test_quantize_overlapping_groups_of_more_than_2_32_blocks():
    """Offsets 0, R, 0, R, ... for 1024 groups: 512 of them hold all R > 2^30 rows, 2^32 + 2560 blocks in all.  Each block
    of the transposed copy is still one group's: the first group's blocks first, then the next one's as far as there
    are columns, no row behind the last one read, nothing written outside.  The first half of the rows holds ones, the
    second twos, and what lies behind x sixty-fours."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    G, C, behind = 1024, 16, 128
    R = 2 ** 30 + 4 * 128 + 77
    B = br.blocks(R)
    half = R // 256 * 128
    assert B * (G // 2) > 2 ** 32 and half % 128 == 0
    T = fd.fp8_block_padded_rows(R, G)
    whole = torch.full((R + behind, C), 64.0, dtype=torch.bfloat16, device=dev)
    whole[:half], whole[half:R] = 1.0, 2.0
    guard = 4096
    codes = torch.full((C * T + 2 * guard,), 0xAA, dtype=torch.uint8, device=dev)
    factors = torch.full((T // 128 * C + 2 * guard,), 7.0, device=dev)
    off = torch.tensor([0, R] * (G // 2) + [0], dtype=torch.int32, device=dev)
    col_q, col_s = codes[guard:-guard].view(C, T), factors[guard:-guard].view(T // 128, C)
    fd.fp8_block_quantize(whole[:R], fd.E4M3, col_q=col_q, col_s=col_s, offsets=off)
    one, two = (1 / (torch.tensor(448.0) / v) for v in (1.0, 2.0))  # fp32: a block's factor
    want = torch.full((T // 128,), one.item(), device=dev)
    want[half // 128:B] = two.item()
    assert T // 128 - B < half // 128  # the second group's blocks that have columns are ones
    assert torch.equal(col_s, want[:, None].expand(-1, C))
    for c in range(C):  # every row is its block's maximum; zeros behind the first group's last row
        assert torch.all(col_q[c, :R] == 0x7E) and torch.all(col_q[c, R:128 * B] == 0) and torch.all(col_q[c, 128 * B:] == 0x7E)
    for t, v in ((codes, 0xAA), (factors, 7.0)):
        assert torch.all(t[:guard] == v) and torch.all(t[-guard:] == v)
    del whole, codes, col_q
    torch.cuda.empty_cache()


def _specials(rows, cols, dtype):
    """Normal values with infinities, NaN, zeros and extremes: single ones, whole lanes of eight, whole blocks of 128."""
    x = wl.normal((rows, cols), 1.0, wl.generator(330, "specials%d" % rows), torch.float32)
    inf, nan = float("inf"), float("nan")
    x[1, 3], x[2, 5] = inf, -inf
    x[3, 7], x[3, 9] = nan, inf               # both in one block
    x[4, 0:8] = nan                            # a thread's eight columns
    x[5, 0:128] = nan                          # a block
    x[6, 0:128], x[6, 11] = nan, 0.5           # all but one
    x[7, 0:128], x[7, 100] = inf, -inf         # nothing finite
    x[8, 0:128] = 0.0
    x[9, 0:128], x[9, 64] = 0.0, nan
    x[10, 0:128], x[10, 64] = -0.0, inf
    x[11, 0:128] = 1e-40                       # subnormal
    x[12, 0:128] = 2.0 ** -101                 # below the floor of the maximum
    x[13, 0:128] = 3e38
    x[14, 0:128] *= 2.0 ** -90
    x[:, 130], x[:, 131] = nan, inf            # whole columns
    x[:, 132] = 0.0
    x[0, 132] = nan
    return x.to(dtype)


def _same(got, want, x, fmt):
    """Codes, where a NaN may have either sign."""
    got, nan = got.cpu().numpy(), np.isnan(x)
    assert np.array_equal(got[~nan], want[~nan])
    assert torch.from_numpy(got[nan]).view(br.F8[fmt]).float().isnan().all()


@pytest.mark.parametrize("groups", [None, [0, 3, 3, 16, 120, 200]])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_specials(dtype, fmt, groups):
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    R, C = 200, 272
    x = _specials(R, C, dtype)
    xf = x.float().numpy()
    G = len(groups) - 1 if groups else 0
    T = fd.fp8_block_padded_rows(R, G)
    row_q, col_q = (torch.full(s, 0xAA, dtype=torch.uint8, device=dev) for s in ((R, C), (C, T)))
    row_s, col_s = torch.full((br.blocks(C), R), 7.0, device=dev), torch.full((T // 128, C), 7.0, device=dev)
    off = torch.tensor(groups, dtype=torch.int32, device=dev) if groups else None
    fd.fp8_block_quantize(x.to(dev), fmt, row_q=row_q, row_s=row_s, col_q=col_q, col_s=col_s, offsets=off)
    q, s = br.rows(xf, fmt)
    qt, st, used = br.cols(xf, fmt, groups)
    _same(row_q, q, xf, fmt)
    assert np.array_equal(row_s.cpu().numpy(), s)
    off = groups or [0, R]
    xt = np.zeros((C, used), np.float32)  # the padded, transposed values
    at = 0
    for lo, hi in zip(off[:-1], off[1:]):
        xt[:, at:at + hi - lo] = xf[lo:hi].T
        at += 128 * br.blocks(hi - lo)
    _same(col_q[:, :used], qt[:, :used], xt, fmt)
    assert np.array_equal(col_s.cpu().numpy()[:used // 128], st[:used // 128])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_weight_specials(dtype, fmt):
    """A block each: one infinity, one NaN, a NaN and an infinity, nothing finite, only NaN, zeros and a NaN, the
    smallest and largest magnitudes."""
    import fp8_delayed_scaling_gb300 as fd
    dev = gpu()
    R, C = 272, 400
    w = wl.normal((2, R, C), 0.02, wl.generator(331, "weight specials"), torch.float32)
    inf, nan = float("inf"), float("nan")
    w[0, 5, 7] = inf
    w[0, 9, 130] = nan
    w[0, 3, 260], w[0, 4, 261] = nan, -inf
    w[0, :128, 384:] = inf
    w[0, 128:256, :128] = nan
    w[0, 128:256, 128:256] = 0.0
    w[0, 200, 200] = nan
    w[0, 128:256, 256:384] = 2.0 ** -120
    w[0, 256:, :128] = 3e38
    w[0, 256:, 128:256], w[0, 270, 140] = -0.0, -inf
    w[1, 271, 399] = nan
    w = w.to(dtype)
    q, q_t = (torch.full(s, 0xAA, dtype=torch.uint8, device=dev) for s in ((2, R, C), (2, C, R)))
    s, s_t = torch.full((2, 4, 3), 7.0, device=dev), torch.full((2, 3, 4), 7.0, device=dev)
    fd.fp8_block_quantize_weight(w.to(dev), fmt, q=q, s=s, q_t=q_t, s_t=s_t)
    for e in range(2):
        wf = w[e].float().numpy()
        rq, rs = br.weight(wf, fmt)
        _same(q[e], rq, wf, fmt)
        _same(q_t[e], np.ascontiguousarray(rq.T), np.ascontiguousarray(wf.T), fmt)
        assert np.array_equal(s[e].cpu().numpy(), rs) and np.array_equal(s_t[e].cpu().numpy(), rs.T)


THREADS = r'''
import threading, torch
import fp8_delayed_scaling_gb300 as fd
dev = torch.device("cuda", 0)
torch.cuda.set_device(dev)
T, G, R, C = 8, 3, 300, 528
g = torch.Generator().manual_seed(11)
xs = [torch.randn(R, C, generator=g).to(torch.bfloat16).to(dev) for _ in range(T)]
w = torch.randn(G, C, C, generator=g).to(dev)
off = torch.tensor([0, 40, 40, 300], dtype=torch.int32, device=dev)
torch.cuda.synchronize()

def work(i, out):
    torch.cuda.set_device(dev)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        u8, f32 = dict(dtype=torch.uint8, device=dev), dict(device=dev)
        P = fd.fp8_block_padded_rows(R, G)
        q, s, qt, st = torch.empty(R, C, **u8), torch.empty(5, R, **f32), torch.zeros(C, P, **u8), torch.zeros(P // 128, C, **f32)
        wq, ws = torch.empty(G, C, C, **u8), torch.empty(G, 5, 5, **f32)
        D, E = torch.empty(R, C, **f32), torch.empty(R, C, **f32)
        W, F = torch.empty(G, C, C, **f32), torch.empty(16, C, **f32)
        fd.fp8_block_quantize_weight(w, fd.E4M3, q=wq, s=ws)
        fd.fp8_block_quantize(xs[i], fd.E4M3, row_q=q, row_s=s, col_q=qt, col_s=st, offsets=off)
        fd.fp8_block_gemm(q, fd.E4M3, s, wq[1], fd.E4M3, ws[1].clone(), D)
        fd.fp8_block_gemm(q[:16], fd.E4M3, s[:, :16].contiguous(), wq[0], fd.E4M3, ws[0], F)
        fd.fp8_block_gemm_grouped(q, fd.E4M3, s, wq, fd.E4M3, ws, off, E)
        fd.fp8_block_gemm_grouped_wgrad(qt, fd.E4M3, st, qt, fd.E4M3, st, off, W)
        stream.synchronize()
        out[i] = [t.cpu() for t in (q, s, qt, st, wq, ws, D, E, W, F)]

first, again = [None] * T, [None] * T
barrier = threading.Barrier(T)
def run(i):
    barrier.wait()
    work(i, first)
ts = [threading.Thread(target=run, args=(i,)) for i in range(T)]
for t in ts: t.start()
for t in ts: t.join()
for i in range(T):
    work(i, again)
for i in range(T):
    assert first[i] is not None, i
    for k, (a, b) in enumerate(zip(first[i], again[i])):
        assert torch.equal(a, b), (i, k)
print("threads ok")
'''


def test_concurrent_first_calls_from_host_threads():
    """A fresh process, eight threads on streams of their own: the set-up of the products runs once under its lock, and
    products on eight streams at once give the bits of a serial rerun."""
    gpu()
    env = dict(os.environ)
    env["PYTHONPATH"] = ROOT + os.pathsep + env.get("PYTHONPATH", "")
    r = subprocess.run([sys.executable, "-c", THREADS], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "threads ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]


def _values(q, fmt, s, per=1):
    return br.values(q, fmt, s, per)


@pytest.mark.parametrize("grad", [0, 1])
@pytest.mark.parametrize("off,rows", [([0, 1, 1, 4], 6), ([3, 40, 40, 95], 97), ([2, 40, 180, 500], 513), ([0, 700, 700, 1500], 1500)],
                         ids=["decode", "tens", "ragged", "many"])
def test_experts_element_by_element(off, rows, grad):
    """Every element of an expert layer's output and gradients, from the same codes, within the product's bound: 16, 32
    and 64 rows a tile and the 256-row tiles."""
    from fp8_delayed_scaling_gb300.blocklinear import BlockExperts
    dev = gpu()
    G, n, k = len(off) - 1, 400, 528
    g = wl.generator(332, "elements%d" % rows)
    x, w = wl.normal((rows, k), 1.0, g, torch.bfloat16), wl.normal((G, n, k), 0.02, g, torch.bfloat16)
    dy = wl.normal((rows, n), 1e-3, g, torch.bfloat16)
    ex = BlockExperts(w.to(dev), rows, out_dtype=torch.float32, grad_dtype=grad)
    y = ex.forward(x.to(dev), torch.tensor(off, dtype=torch.int32, device=dev))
    dx, dw = ex.backward(dy.to(dev))
    xf, df = x.float().numpy(), dy.float().numpy()
    xv, dv = _values(*_with(br.rows(xf, 0), 0)), _values(*_with(br.rows(df, grad), grad))
    xt, xs, _ = br.cols(xf, 0, off)
    dt, ds, _ = br.cols(df, grad, off)
    at = 0
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        wq, wsc = br.weight(w[e].float().numpy(), 0)
        wv = _values(wq, 0, wsc, 128)
        b = br.blocks(hi - lo)
        a, c = (_values(q[:, at:at + 128 * b], f, s[at // 128:at // 128 + b]) for q, f, s in ((dt, grad, ds), (xt, 0, xs)))
        br.check(dw[e], a @ c.T, np.abs(a) @ np.abs(c).T, 128 * b, "dw of group %d" % e)
        at += 128 * b
        if lo == hi:
            continue
        br.check(y[lo:hi], xv[lo:hi] @ wv.T, np.abs(xv[lo:hi]) @ np.abs(wv).T, k, "y of group %d" % e)
        br.check(dx[lo:hi], dv[lo:hi] @ wv, np.abs(dv[lo:hi]) @ np.abs(wv), n, "dx of group %d" % e)


def _with(codes, fmt):
    return codes[0], fmt, codes[1]
