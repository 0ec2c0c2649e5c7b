"""Block-scaled FP8 (one fp32 scale per 128 values) on the GPU, against plain numpy: codes and
factors bit for bit, products within the bound that block_reference.bound derives."""
import numpy as np
import pytest
import torch

import block_reference as br
import workloads as wl
from helpers import gpu

pytestmark = pytest.mark.gpu


def _fd():
    import fp8_delayed_scaling_gb300 as fd
    return fd, gpu()


def _x(rows, cols, dtype, name):
    """Normal values over many magnitudes per column, with zero and special blocks."""
    g = wl.generator(300, name)
    ch = torch.exp2(torch.randint(-12, 12, (cols,), generator=g).float())
    return (torch.randn((rows, cols), generator=g) * ch).to(dtype)


def _buffers(fd, rows, cols, groups, dev):
    T = fd.fp8_block_padded_rows(rows, groups)
    fill = dict(device=dev)
    return dict(row_q=torch.full((rows, cols), 0xAA, dtype=torch.uint8, **fill),
                row_s=torch.full((br.blocks(cols), rows), 7.0, **fill),
                col_q=torch.full((cols, T), 0xAA, dtype=torch.uint8, **fill),
                col_s=torch.full((T // 128, cols), 7.0, **fill))


QUANT = [(1, 16), (5, 128), (127, 144), (128, 256), (129, 112), (300, 400), (1, 4096), (1000, 48)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("rows,cols", QUANT)
def test_quantize(rows, cols, fmt, dtype):
    fd, dev = _fd()
    x = _x(rows, cols, dtype, "q%d.%d" % (rows, cols))
    x[:, :16] = 0  # short zero runs, and whole zero blocks where the matrix is narrow
    b = _buffers(fd, rows, cols, 0, dev)
    db = torch.full((cols,), 7.0, device=dev)
    ws = torch.empty(fd.fp8_cast_workspace_size(rows, cols), dtype=torch.uint8, device=dev)
    fd.fp8_block_quantize(x.to(dev), fmt, dbias=db, workspace=ws, **b)
    xf = x.float().numpy()
    q, s = br.rows(xf, fmt)
    qt, st, _ = br.cols(xf, fmt)
    assert np.array_equal(b["row_q"].cpu().numpy(), q) and np.array_equal(b["row_s"].cpu().numpy(), s)
    assert np.array_equal(b["col_q"].cpu().numpy(), qt) and np.array_equal(b["col_s"].cpu().numpy(), st)
    # fp32 sums of `rows` terms in a tree or in order: at most rows roundings of 2^-24
    assert np.all(np.abs(db.cpu().numpy() - xf.astype(np.float64).sum(0)) <= rows * 2.0 ** -24 * np.abs(xf).sum(0))
    one = _buffers(fd, rows, cols, 0, dev)  # either direction alone gives the same bits
    fd.fp8_block_quantize(x.to(dev), fmt, row_q=one["row_q"], row_s=one["row_s"])
    fd.fp8_block_quantize(x.to(dev), fmt, col_q=one["col_q"], col_s=one["col_s"])
    for k in one:
        assert torch.equal(one[k], b[k]), k


@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize_special_values(fmt):
    """Infinities saturate, NaN stays, neither enters a block's maximum; the smallest and largest magnitudes."""
    fd, dev = _fd()
    x = _x(256, 256, torch.float32, "special")
    x[3, 5], x[4, 200], x[130, 7] = float("inf"), float("-inf"), float("nan")
    x[7] = 0.0
    x[7, 9] = float("inf")        # nothing finite but zeros
    x[8] = 1e-42                  # subnormal
    x[9] = 2.0 ** -101            # below the floor of the maximum
    x[10] = 3.4e38
    x[:, 128:] *= 2.0 ** -60
    b = _buffers(fd, 256, 256, 0, dev)
    fd.fp8_block_quantize(x.to(dev), fmt, **b)
    xf = x.numpy()
    q, s = br.rows(xf, fmt)
    qt, st, _ = br.cols(xf, fmt)
    nan = np.isnan(xf)
    got, got_t = b["row_q"].cpu().numpy(), b["col_q"].cpu().numpy()
    assert np.array_equal(got[~nan], q[~nan]) and np.array_equal(got_t[~nan.T], qt[~nan.T])
    for codes, where in ((got, nan), (got_t, nan.T)):
        assert torch.from_numpy(codes[where]).view(br.F8[fmt]).float().isnan().all()
    assert np.array_equal(b["row_s"].cpu().numpy(), s) and np.array_equal(b["col_s"].cpu().numpy(), st)


GROUPS = [[0, 5], [0, 0, 128, 128, 129, 300], [3, 130, 131, 131, 400], [0] * 40 + [1], list(range(0, 129, 2)),
          [0, 256, 256 + 127, 700], [17, 17, 17]]


@pytest.mark.parametrize("off", GROUPS, ids=range(len(GROUPS)))
def test_quantize_groups(off):
    fd, dev = _fd()
    rows, cols, fmt = off[-1] + 37, 272, 0
    x = _x(rows, cols, torch.bfloat16, "g%s" % off[:6])
    b = _buffers(fd, rows, cols, len(off) - 1, dev)
    fd.fp8_block_quantize(x.to(dev), fmt, offsets=torch.tensor(off, dtype=torch.int32, device=dev), **b)
    xf = x.float().numpy()
    q, s = br.rows(xf, fmt)
    qt, st, used = br.cols(xf, fmt, off)
    inside = slice(off[0], off[-1])
    got = {k: v.cpu().numpy() for k, v in b.items()}
    assert np.array_equal(got["row_q"][inside], q[inside]) and np.array_equal(got["row_s"][:, inside], s[:, inside])
    assert np.all(got["row_q"][:off[0]] == 0xAA) and np.all(got["row_q"][off[-1]:] == 0xAA)
    assert np.all(got["row_s"][:, :off[0]] == 7.0) and np.all(got["row_s"][:, off[-1]:] == 7.0)
    assert np.array_equal(got["col_q"][:, :used], qt[:, :used]) and np.all(got["col_q"][:, used:] == 0xAA)
    assert np.array_equal(got["col_s"][:used // 128], st[:used // 128]) and np.all(got["col_s"][used // 128:] == 7.0)


SHORT = [[0, 1, 17, 33, 65, 66, 129, 290], [4] + [4 + 3 * i for i in range(1, 300)], list(range(0, 1025)),
         [0, 16, 32, 64, 128, 256, 256]]


@pytest.mark.parametrize("dtype,fmt", [(torch.bfloat16, 1), (torch.float32, 0)])
@pytest.mark.parametrize("off", SHORT, ids=range(len(SHORT)))
def test_quantize_short_groups(off, dtype, fmt):
    """Groups of a few rows share a block of threads between column tiles; eleven of those, the last one narrow."""
    fd, dev = _fd()
    rows, cols = off[-1] + 3, 1296
    x = _x(rows, cols, dtype, "s%s" % off[:6])
    x[off[0] + 1, 600] = float("inf")
    b = _buffers(fd, rows, cols, len(off) - 1, dev)
    o = torch.tensor(off, dtype=torch.int32, device=dev)
    fd.fp8_block_quantize(x.to(dev), fmt, offsets=o, **b)
    xf = x.float().numpy()
    q, s = br.rows(xf, fmt)
    qt, st, used = br.cols(xf, fmt, off)
    inside = slice(off[0], off[-1])
    got = {k: v.cpu().numpy() for k, v in b.items()}
    assert np.array_equal(got["row_q"][inside], q[inside]) and np.array_equal(got["row_s"][:, inside], s[:, inside])
    assert np.array_equal(got["col_q"][:, :used], qt[:, :used]) and np.all(got["col_q"][:, used:] == 0xAA)
    assert np.array_equal(got["col_s"][:used // 128], st[:used // 128]) and np.all(got["col_s"][used // 128:] == 7.0)
    one = _buffers(fd, rows, cols, len(off) - 1, dev)  # either direction alone: the same bits, the same rows left alone
    fd.fp8_block_quantize(x.to(dev), fmt, row_q=one["row_q"], row_s=one["row_s"], offsets=o)
    fd.fp8_block_quantize(x.to(dev), fmt, col_q=one["col_q"], col_s=one["col_s"], offsets=o)
    for k in one:
        assert torch.equal(one[k], b[k]), k


def test_quantize_wrong_offsets_stay_inside():
    """Offsets in disorder or behind the last row give wrong codes, and no access outside the tensors."""
    fd, dev = _fd()
    rows, cols, off = 300, 272, [7, 900, 100, -5, 250, 5000, -2 ** 31, 2 ** 31 - 1]
    x = _x(rows, cols, torch.bfloat16, "wrong").to(dev)
    T = fd.fp8_block_padded_rows(rows, len(off) - 1)
    sizes = dict(row_q=(torch.uint8, (rows, cols)), row_s=(torch.float32, (br.blocks(cols), rows)),
                 col_q=(torch.uint8, (cols, T)), col_s=(torch.float32, (T // 128, cols)))
    whole = {k: torch.full((shape[0] * shape[1] + 8192,), 7, dtype=t, device=dev) for k, (t, shape) in sizes.items()}
    view = {k: whole[k][4096:-4096].view(shape) for k, (t, shape) in sizes.items()}
    fd.fp8_block_quantize(x, 0, offsets=torch.tensor(off, dtype=torch.int32, device=dev), **view)
    for v in whole.values():
        assert torch.all(v[:4096] == 7) and torch.all(v[-4096:] == 7)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(16, 16), (128, 128), (144, 400), (1, 1008, 272), (5, 48, 1040)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize_weight(shape, fmt, dtype):
    fd, dev = _fd()
    R, C = shape[-2:]
    lead = shape[:-2]
    w = _x((lead[0] if lead else 1) * R, C, dtype, "w%s" % (shape,)).view(shape)
    w.view(-1, C)[:, 0] = 0
    q = torch.full(shape, 0xAA, dtype=torch.uint8, device=dev)
    s = torch.full(lead + (br.blocks(C), br.blocks(R)), 7.0, device=dev)
    q_t = torch.full(lead + (C, R), 0xAA, dtype=torch.uint8, device=dev)
    s_t = torch.full(lead + (br.blocks(R), br.blocks(C)), 7.0, device=dev)
    fd.fp8_block_quantize_weight(w.to(dev), fmt, q=q, s=s, q_t=q_t, s_t=s_t)
    for e in range(lead[0] if lead else 1):
        at = (e,) if lead else ()
        rq, rs = br.weight(w[at].float().numpy(), fmt)
        assert np.array_equal(q[at].cpu().numpy(), rq) and np.array_equal(s[at].cpu().numpy(), rs)
        assert np.array_equal(q_t[at].cpu().numpy(), rq.T) and np.array_equal(s_t[at].cpu().numpy(), rs.T)


# ---------------------------------------------------------------------------------------------- products
def _operand(rows, K, fmt, name, per=1):
    x = _x(rows, K, torch.float32, name).numpy()
    return br.rows(x, fmt) if per == 1 else br.weight(x, fmt)


def _dev(dev, *arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).to(dev) for a in arrays]


GEMMS = [  # M, N, K, fmt_a, b per row, bias dtype, D dtype
    (1, 16, 16, 0, False, None, torch.float32),
    (1, 4096, 4096, 0, False, torch.bfloat16, torch.bfloat16),
    (2, 272, 1040, 0, False, None, torch.float32),
    (7, 1008, 2048, 1, False, torch.float32, torch.bfloat16),
    (16, 128, 8192, 0, False, None, torch.float32),
    (17, 144, 128, 0, False, torch.bfloat16, torch.float32),
    (31, 2048, 144, 0, False, None, torch.bfloat16),
    (33, 512, 512, 1, False, None, torch.float32),
    (64, 640, 4112, 0, False, torch.float32, torch.float32),
    (65, 400, 1024, 0, False, None, torch.bfloat16),
    (128, 256, 2048, 0, False, None, torch.float32),
    (129, 272, 384, 0, False, torch.bfloat16, torch.float32),
    (300, 784, 1040, 1, False, None, torch.bfloat16),
    (257, 16, 16, 0, False, None, torch.float32),
    (1000, 1040, 272, 0, False, torch.float32, torch.bfloat16),
    (1, 16, 128, 0, True, None, torch.float32),
    (48, 400, 4096, 1, True, None, torch.float32),
    (272, 1008, 1040, 0, True, torch.bfloat16, torch.bfloat16),
    (640, 528, 384, 1, True, None, torch.float32),
    (20000, 48, 256, 0, False, None, torch.float32),
    # few tiles and a long reduction: pairs share a tile's blocks (uneven shares, ragged rows and columns)
    (600, 1040, 4112, 0, False, torch.bfloat16, torch.bfloat16),
    (700, 2064, 3088, 1, False, torch.float32, torch.float32),
    (300, 528, 6160, 0, True, torch.bfloat16, torch.float32),
    (513, 1296, 4240, 1, True, None, torch.bfloat16),
    # a weight tile's blocks over three, four, five and six CTAs (uneven shares, ragged rows)
    (19, 6016, 528, 0, False, torch.float32, torch.float32),
    (61, 4096, 1168, 1, False, None, torch.bfloat16),
    (50, 3600, 1424, 0, False, torch.bfloat16, torch.bfloat16),
    (9, 1040, 2576, 0, False, torch.bfloat16, torch.float32),
    # more tiles than run at once
    (2500, 2064, 400, 0, False, torch.bfloat16, torch.float32),
    (2310, 2320, 256, 1, True, torch.float32, torch.bfloat16),
    # and a long reduction: the tiles left at the end are shared
    (1290, 3344, 5520, 0, False, torch.float32, torch.bfloat16),
    (1100, 4112, 5648, 1, True, torch.bfloat16, torch.float32),
]


@pytest.mark.parametrize("M,N,K,fa,brows,bias,dtype", GEMMS)
def test_gemm(M, N, K, fa, brows, bias, dtype):
    fd, dev = _fd()
    a, a_s = _operand(M, K, fa, "a%d" % M)
    b, b_s = _operand(N, K, 0, "b%d" % N, 1 if brows else 128)
    av, bv = br.values(a, fa, a_s, 1), br.values(b, 0, b_s, 1 if brows else 128)
    ref, absum = av @ bv.T, np.abs(av) @ np.abs(bv).T
    D = torch.full((M, N), 7.0, dtype=dtype, device=dev)
    t = _dev(dev, a, a_s, b, b_s)
    bt = None
    if bias is not None:
        bt = wl.normal((N,), float(np.abs(ref).mean()), wl.generator(301, "bias"), bias).to(dev)
        ref = ref + bt.double().cpu().numpy()
        absum = absum + np.abs(bt.double().cpu().numpy())
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    fd.fp8_block_gemm(t[0], fa, t[1], t[2], 0, t[3], D, bias=bt, dev_status=status)
    br.check(D, ref, absum, K, "gemm")
    assert status.item() == 0
    again = torch.full_like(D, 9.0)
    fd.fp8_block_gemm(t[0], fa, t[1], t[2], 0, t[3], again, bias=bt)
    assert torch.equal(D, again)  # the same bits on every call


def test_gemm_nan_code_stays_in_its_row():
    fd, dev = _fd()
    a, a_s = _operand(200, 512, 0, "nan")
    b, b_s = _operand(256, 512, 0, "nan_b", 128)
    a[77, 300] = 0x7F
    t = _dev(dev, a, a_s, b, b_s)
    D = torch.empty((200, 256), device=dev)
    fd.fp8_block_gemm(t[0], 0, t[1], t[2], 0, t[3], D)
    bad = D.isnan().any(1).cpu()
    assert bad[77] and bad.sum() == 1 and D[77].isnan().all()


ROWS = [  # offsets, rows, N, K, D dtype
    ([0, 1], 1, 16, 16, torch.float32),
    ([0, 0, 3, 3, 4], 9, 272, 400, torch.float32),
    ([0, 1, 1, 2, 5, 16], 16, 512, 1024, torch.bfloat16),
    ([0] * 30 + [2, 2, 7], 8, 144, 512, torch.float32),
    ([5, 37, 100, 100, 228], 240, 384, 272, torch.bfloat16),
    ([0, 256, 256, 513, 1000], 1000, 528, 640, torch.float32),
    ([0, 700, 701, 1500], 1531, 1040, 256, torch.bfloat16),
    ([3, 3, 3], 10, 64, 128, torch.float32),
    (list(range(0, 1025)), 1024, 48, 128, torch.float32),
]


@pytest.mark.parametrize("off,rows,N,K,dtype", ROWS, ids=range(len(ROWS)))
def test_grouped(off, rows, N, K, dtype):
    fd, dev = _fd()
    G = len(off) - 1
    a, a_s = _operand(rows, K, 0, "ga%d" % rows)
    qs = [_operand(N, K, 0, "gb%d" % e, 128) for e in range(min(G, 8))]
    b, b_s = np.stack([qs[e % 8][0] for e in range(G)]), np.stack([qs[e % 8][1] for e in range(G)])
    av = br.values(a, 0, a_s, 1)
    D = torch.full((rows, N), 7.0, dtype=dtype, device=dev)
    t = _dev(dev, a, a_s, b, b_s)
    o = torch.tensor(off, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    fd.fp8_block_gemm_grouped(t[0], 0, t[1], t[2], 0, t[3], o, D, dev_status=status)
    assert status.item() == 0
    ref, absum = np.full((rows, N), 7.0), np.zeros((rows, N))
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        if hi > lo:
            bv = br.values(b[e], 0, b_s[e], 128)
            ref[lo:hi], absum[lo:hi] = av[lo:hi] @ bv.T, np.abs(av[lo:hi]) @ np.abs(bv).T
    br.check(D, ref, absum, K, "grouped")
    assert torch.all(D[:off[0]] == 7.0) and torch.all(D[off[-1]:] == 7.0)  # rows outside the groups as they were


REDUCE = [  # offsets, rows, M, N, D dtype
    ([0, 1], 1, 16, 16, torch.float32),
    ([0, 0, 3, 3, 4], 9, 272, 400, torch.float32),
    ([0, 128, 257, 257, 700], 700, 256, 528, torch.bfloat16),
    ([5, 37, 100, 100, 228], 240, 300, 48, torch.float32),
    ([0] * 30 + [2, 2, 7], 8, 144, 64, torch.float32),
    ([2, 2], 5, 64, 32, torch.bfloat16),
]


@pytest.mark.parametrize("off,rows,M,N,dtype", REDUCE, ids=range(len(REDUCE)))
def test_grouped_wgrad(off, rows, M, N, dtype):
    fd, dev = _fd()
    G = len(off) - 1
    o = torch.tensor(off, dtype=torch.int32, device=dev)
    ops = []
    for name, cols, fmt in (("dy", M, 1), ("x", N, 0)):
        x = _x(rows, br.blocks(cols) * 128, torch.float32, "wg%s%d" % (name, cols))[:, :cols].contiguous()
        q, s, used = br.cols(x.numpy(), fmt, off)
        q[:, used:] = 0x7F  # never read: NaN codes there must not show
        s[used // 128:] = np.nan
        ops += [q, s]
    t = _dev(dev, *ops)
    D = torch.full((G, M, N), 7.0, dtype=dtype, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    fd.fp8_block_gemm_grouped_wgrad(t[0], 1, t[1], t[2], 0, t[3], o, D, dev_status=status)
    assert status.item() == 0
    at = 0
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        n = br.blocks(hi - lo)
        av = br.values(ops[0][:, at:at + 128 * n], 1, ops[1][at // 128:at // 128 + n], 1)
        bv = br.values(ops[2][:, at:at + 128 * n], 0, ops[3][at // 128:at // 128 + n], 1)
        br.check(D[e], av @ bv.T, np.abs(av) @ np.abs(bv).T, 128 * n, "wgrad of group %d" % e)
        if hi == lo:
            assert torch.all(D[e] == 0.0)
        at += 128 * n


def test_grouped_wgrad_with_mostly_empty_groups():
    """More tiles than the GPU runs at once, most of them of groups without rows, and the rest one or two blocks long."""
    fd, dev = _fd()
    G, M, N = 1000, 256, 272
    rng = np.random.default_rng(9)
    lens = np.where(rng.random(G) < 0.12, rng.integers(1, 200, G), 0)
    off = np.concatenate([[0], np.cumsum(lens)])
    rows = int(off[-1])
    o = torch.tensor(off, dtype=torch.int32, device=dev)
    ops = []
    for cols, fmt in ((M, 1), (N, 0)):
        q, s, _ = br.cols(_x(rows, cols, torch.float32, "sparse%d" % cols).numpy(), fmt, off)
        ops += [q, s]
    t = _dev(dev, *ops)
    D = torch.full((G, M, N), 7.0, device=dev)
    fd.fp8_block_gemm_grouped_wgrad(t[0], 1, t[1], t[2], 0, t[3], o, D)
    at = 0
    for e in range(G):
        n = br.blocks(int(lens[e]))
        if n == 0:
            assert torch.all(D[e] == 0.0)
            continue
        av = br.values(ops[0][:, at:at + 128 * n], 1, ops[1][at // 128:at // 128 + n], 1)
        bv = br.values(ops[2][:, at:at + 128 * n], 0, ops[3][at // 128:at // 128 + n], 1)
        br.check(D[e], av @ bv.T, np.abs(av) @ np.abs(bv).T, 128 * n, "wgrad of group %d" % e)
        at += 128 * n


@pytest.mark.parametrize("rows", [40, 900])  # the kernels for few and for many rows a group
def test_grouped_products_wrong_offsets_stay_inside(rows):
    fd, dev = _fd()
    off, N, K = torch.tensor([7, 600, 100, -5, 250, 5000, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device=dev), 272, 400
    G = off.numel() - 1
    a, a_s = _operand(rows, K, 0, "wa")
    b, b_s = _operand(G * N, K, 0, "wb")
    t = _dev(dev, a, a_s, b)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    whole = torch.full((rows * N + 8192,), 7.0, device=dev)
    fd.fp8_block_gemm_grouped(t[0], 0, t[1], t[2].view(G, N, K), 0, torch.ones((G, br.blocks(K), br.blocks(N)), device=dev), off,
                              whole[4096:-4096].view(rows, N), dev_status=status)
    T = fd.fp8_block_padded_rows(rows, G)
    A, B = (torch.full((n, T), 0x38, dtype=torch.uint8, device=dev) for n in (144, N))
    grads = torch.full((G * 144 * N + 8192,), 7.0, device=dev)
    fd.fp8_block_gemm_grouped_wgrad(A, 0, torch.ones((T // 128, 144), device=dev), B, 0, torch.ones((T // 128, N), device=dev), off,
                                    grads[4096:-4096].view(G, 144, N), dev_status=status)
    for v in (whole, grads):
        assert torch.all(v[:4096] == 7) and torch.all(v[-4096:] == 7)
    assert status.item() == 0


@pytest.mark.parametrize("M,N,K", [(50, 3600, 1424), (600, 1040, 4112), (1100, 4112, 5648), (2500, 2064, 400)])
def test_products_in_order_and_captured(M, N, K):
    """A chain of quantisation, product and a reader of D on one stream, each launch behind the one before it; then the same
    chain replayed from a graph over changed inputs.  Products in one launch, shared ones, and one of two launches."""
    fd, dev = _fd()
    b, b_s = _operand(N, K, 0, "chain", 128)
    b, b_s = _dev(dev, b, b_s)
    x = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    q, s = torch.empty((M, K), dtype=torch.uint8, device=dev), torch.empty((br.blocks(K), M), device=dev)
    D, out = (torch.empty((M, N), dtype=torch.bfloat16, device=dev) for _ in range(2))
    xs = [_x(M, K, torch.bfloat16, "chain%d" % i).to(dev) for i in range(3)]

    def chain(src):
        x.copy_(src)
        fd.fp8_block_quantize(x, 0, row_q=q, row_s=s)
        fd.fp8_block_gemm(q, 0, s, b, 0, b_s, D)
        out.copy_(D)
        D.fill_(7.0)

    want = []
    for src in xs:  # with a wait after every step
        x.copy_(src)
        torch.cuda.synchronize()
        fd.fp8_block_quantize(x, 0, row_q=q, row_s=s)
        torch.cuda.synchronize()
        fd.fp8_block_gemm(q, 0, s, b, 0, b_s, D)
        torch.cuda.synchronize()
        want.append(D.clone())
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for _ in range(3):
            for src, w in zip(xs, want):
                chain(src)
                assert torch.equal(out, w)
        src = xs[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            chain(src)
        for new, w in zip(xs[::-1], want[::-1]):
            src.copy_(new)
            graph.replay()
            assert torch.equal(out, w)
