"""Every way a block-scaled product can run: each case names what fp8_block_gemm_plan must answer for it on a GB300 of
152 SMs (rows of A a tile, how many CTAs or CTA pairs share a tile, whether there are whole and shared tiles), so that a
changed rule of choice shows here and not as a path that nothing tests.  Both FP8 types on both sides."""
import numpy as np
import pytest
import torch

import block_reference as br
import workloads as wl
from helpers import gpu
from test_gpu_block import _dev, _operand

pytestmark = pytest.mark.gpu


def _fd():
    import fp8_delayed_scaling_gb300 as fd
    return fd, gpu()


def _expect(got, want, dev):
    """The choice, where the sizes were made for this many SMs; the results are compared on any number."""
    if torch.cuda.get_device_properties(dev).multi_processor_count == 152:
        assert got == want


DENSE = [  # M, N, K; rows a tile, shares, whole tiles?, shared tiles?; codes of A and B; bias, D
    (5, 688, 144, (16, 1, True, False), 0, 1, torch.bfloat16, torch.float32),
    (13, 1104, 592, (16, 2, False, True), 1, 1, None, torch.bfloat16),
    (21, 1040, 784, (16, 3, False, True), 0, 0, torch.float32, torch.float32),
    (7, 2064, 1040, (16, 4, False, True), 1, 0, torch.bfloat16, torch.bfloat16),
    (30, 1296, 1296, (16, 5, False, True), 0, 1, None, torch.float32),
    (9, 1040, 2576, (16, 6, False, True), 0, 0, torch.bfloat16, torch.bfloat16),
    (1223, 656, 400, (32, 1, True, False), 0, 1, torch.float32, torch.bfloat16),
    (33, 4432, 1552, (32, 2, False, True), 1, 0, None, torch.float32),
    (50, 4944, 656, (32, 3, False, True), 0, 0, torch.bfloat16, torch.bfloat16),
    (19, 4112, 3376, (32, 4, False, True), 1, 1, torch.float32, torch.float32),
    (18, 3216, 2320, (32, 5, False, True), 0, 0, None, torch.bfloat16),
    (633, 48, 5216, (32, 6, False, True), 0, 1, torch.bfloat16, torch.float32),
    (276, 5040, 2976, (64, 1, True, False), 0, 1, torch.bfloat16, torch.float32),
    (67, 4288, 3216, (64, 2, False, True), 1, 0, torch.float32, torch.bfloat16),
    (97, 5712, 1040, (64, 3, False, True), 0, 1, None, torch.float32),
    (39, 3248, 5072, (64, 5, False, True), 0, 0, torch.bfloat16, torch.bfloat16),
    (1040, 2336, 144, (256, 1, True, False), 0, 1, torch.float32, torch.float32),
    (267, 3904, 2992, (256, 2, False, True), 0, 0, torch.bfloat16, torch.bfloat16),
    (1229, 400, 5072, (256, 4, False, True), 1, 1, torch.bfloat16, torch.float32),
    (1801, 2992, 8208, (256, 2, True, True), 0, 1, None, torch.bfloat16),
    (1290, 3344, 5520, (256, 4, True, True), 0, 0, torch.float32, torch.float32),
]
ROWS = [  # the same with factors per row of B
    (272, 1008, 1040, (256, 1, True, False), 0, 1, torch.bfloat16, torch.bfloat16),
    (700, 2064, 3088, (256, 2, False, True), 1, 1, torch.float32, torch.float32),
    (300, 528, 6160, (256, 4, False, True), 0, 1, None, torch.bfloat16),
    (1801, 2992, 8208, (256, 2, True, True), 1, 0, torch.bfloat16, torch.float32),
    (1100, 4112, 5648, (256, 4, True, True), 0, 0, torch.bfloat16, torch.bfloat16),
]


def _values(q, fmt, s, per, dev):
    """block_reference.values on the GPU, in fp64."""
    v = torch.from_numpy(q).to(dev).view(br.F8[fmt]).double()
    f = torch.from_numpy(s).to(dev).double().t().repeat_interleave(per, 0)[:v.shape[0]]
    return v * f.repeat_interleave(128, 1)[:, :v.shape[1]]


@pytest.mark.parametrize("M,N,K,plan,fa,fb,bias,dtype,per", [c + (128,) for c in DENSE] + [c + (1,) for c in ROWS])
def test_product(M, N, K, plan, fa, fb, bias, dtype, per):
    fd, dev = _fd()
    rows, shares, whole, shared = fd.fp8_block_gemm_plan(M, N, K, b_rows=per)
    _expect((rows, shares, whole > 0, shared > 0), plan, dev)
    launches = (whole > 0) + (shared > 0)
    a, a_s = _operand(M, K, fa, "pa%d" % M)
    b, b_s = _operand(N, K, fb, "pb%d" % N, per)
    av, bv = _values(a, fa, a_s, 1, dev), _values(b, fb, b_s, per, dev)
    ref, absum = av @ bv.t(), av.abs() @ bv.abs().t()
    bt = None
    if bias is not None:
        bt = wl.normal((N,), float(ref.abs().mean()), wl.generator(301, "plan bias"), bias).to(dev)
        ref, absum = ref + bt.double(), absum + bt.double().abs()
    t = _dev(dev, a, a_s, b, b_s)
    around = torch.full((M * N + 8192,), 7.0, dtype=dtype, device=dev)
    D = around[4096:-4096].view(M, N)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    n0 = fd.fp8dl_kernel_launches()
    fd.fp8_block_gemm(t[0], fa, t[1], t[2], fb, t[3], D, bias=bt, dev_status=status)
    assert fd.fp8dl_kernel_launches() - n0 == launches
    br.check(D, ref.cpu().numpy(), absum.cpu().numpy(), K, "gemm")
    assert status.item() == 0
    assert torch.all(around[:4096] == 7) and torch.all(around[-4096:] == 7)
    again = torch.full_like(D, 9.0)
    fd.fp8_block_gemm(t[0], fa, t[1], t[2], fb, t[3], again, bias=bt)
    assert torch.equal(D, again)


GROUPED = [  # groups, rows, N, K; rows a tile, CTAs a weight tile; codes of A and B; D
    (4, 60, 400, 272, (16, 1), 0, 1, torch.float32),
    (3, 45, 272, 400, (16, 2), 1, 0, torch.bfloat16),
    (3, 45, 144, 784, (16, 3), 1, 1, torch.float32),
    (2, 31, 272, 1040, (16, 4), 0, 0, torch.bfloat16),
    (2, 31, 272, 1296, (16, 5), 0, 1, torch.float32),
    (2, 32, 144, 1568, (16, 6), 1, 0, torch.float32),
    (4, 130, 1040, 272, (32, 1), 0, 1, torch.bfloat16),
    (4, 150, 144, 448, (32, 2), 1, 0, torch.float32),
    (3, 110, 144, 784, (32, 3), 0, 0, torch.bfloat16),
    (3, 130, 272, 1040, (32, 4), 1, 1, torch.float32),
    (2, 70, 272, 1296, (32, 5), 0, 1, torch.bfloat16),
    (3, 120, 144, 1552, (32, 6), 0, 0, torch.float32),
    (5, 365, 272, 144, (64, 1), 1, 0, torch.float32),
    (4, 300, 144, 400, (64, 2), 0, 1, torch.bfloat16),
    (3, 230, 144, 784, (64, 3), 0, 0, torch.float32),
    (3, 220, 272, 1040, (64, 4), 1, 1, torch.bfloat16),
    (3, 200, 272, 1296, (64, 5), 0, 1, torch.float32),
    (2, 150, 144, 1552, (64, 6), 1, 0, torch.bfloat16),
    (9, 400, 2064, 528, (32, 1), 1, 0, torch.bfloat16),   # more tiles than CTAs at once
    (5, 1300, 1040, 400, (256, 1), 1, 0, torch.float32),
    (3, 900, 272, 656, (256, 1), 0, 1, torch.bfloat16),
    (3, 1000, 528, 272, (256, 1), 1, 1, torch.bfloat16),
]


def _offsets(G, rows):
    """Two rows before the first group, three behind the last one; the second group (of three or more) is idle, the last
    one long (several tiles), the others short."""
    lens = [0 if G > 2 and g == 1 else 1 + rows // (4 * G) + g for g in range(G - 1)]
    return [2] + [2 + sum(lens[:g + 1]) for g in range(G - 1)] + [rows - 3]


def test_plan_names_shares_only_where_tiles_are_shared():
    """Tiles that fill the pairs exactly leave none to share, however long the reduction; and sizes of all kinds."""
    fd, dev = _fd()
    _expect(fd.fp8_block_gemm_plan(19 * 256, 4 * 256, 8192), (256, 1, 76, 0), dev)
    rng = np.random.default_rng(17)
    for _ in range(2000):
        M, N, K = (int(np.exp(rng.uniform(0, np.log(v)))) for v in (20000, 800, 800))
        groups = int(rng.integers(0, 2) * rng.integers(1, 100))
        rows, shares, whole, shared = fd.fp8_block_gemm_plan(M, 16 * N, 16 * K, n_groups=groups)
        assert rows in (16, 32, 64, 256) and whole >= 0 and shared >= 0 and whole + shared > 0
        assert (shares > 1) == (shared > 0) and 1 <= shares <= (4 if rows == 256 else 6)


@pytest.mark.parametrize("G,rows,N,K,plan,fa,fb,dtype", GROUPED)
def test_grouped(G, rows, N, K, plan, fa, fb, dtype):
    fd, dev = _fd()
    got = fd.fp8_block_gemm_plan(rows, N, K, n_groups=G)
    _expect(got[:2], plan, dev)
    assert (got[2] == 0) == (got[1] > 1) and (got[3] > 0) == (got[1] > 1)
    off = _offsets(G, rows)
    assert off[-1] - off[-2] > plan[0] and (G == 2 or off[1] == off[2])
    a, a_s = _operand(rows, K, fa, "pga%d" % rows)
    ws = [_operand(N, K, fb, "pgb%d" % e, 128) for e in range(G)]
    b, b_s = np.stack([w[0] for w in ws]), np.stack([w[1] for w in ws])
    t = _dev(dev, a, a_s, b, b_s)
    D = torch.full((rows, N), 7.0, dtype=dtype, device=dev)
    o = torch.tensor(off, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    fd.fp8_block_gemm_grouped(t[0], fa, t[1], t[2], fb, t[3], o, D, dev_status=status)
    ref, absum = np.full((rows, N), 7.0), np.zeros((rows, N))
    av = br.values(a, fa, a_s, 1)
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        bv = br.values(b[e], fb, b_s[e], 128)
        ref[lo:hi], absum[lo:hi] = av[lo:hi] @ bv.T, np.abs(av[lo:hi]) @ np.abs(bv).T
    br.check(D, ref, absum, K, "grouped")
    assert status.item() == 0
    assert torch.all(D[:off[0]] == 7.0) and torch.all(D[off[-1]:] == 7.0)
    again = torch.full_like(D, 7.0)
    fd.fp8_block_gemm_grouped(t[0], fa, t[1], t[2], fb, t[3], o, again)
    assert torch.equal(D, again)


@pytest.mark.parametrize("fa,fb", [(0, 1), (1, 1), (0, 0)])
def test_grouped_wgrad_types(fa, fb):
    """The types of both operands; groups of none, a few and several blocks."""
    fd, dev = _fd()
    off, M, N = [1, 1, 60, 188, 700], 300, 272
    ops = []
    for cols, fmt in ((M, fa), (N, fb)):
        x = wl.normal((off[-1] + 2, cols), 1.0, wl.generator(302, "wg%d" % cols)).numpy()
        ops += list(br.cols(x, fmt, off)[:2])
    t = _dev(dev, *ops)
    D = torch.full((4, M, N), 7.0, device=dev)
    fd.fp8_block_gemm_grouped_wgrad(t[0], fa, t[1], t[2], fb, t[3], torch.tensor(off, dtype=torch.int32, device=dev), D)
    at = 0
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        n = br.blocks(hi - lo)
        av = br.values(ops[0][:, at:at + 128 * n], fa, ops[1][at // 128:at // 128 + n], 1)
        bv = br.values(ops[2][:, at:at + 128 * n], fb, ops[3][at // 128:at // 128 + n], 1)
        br.check(D[e], av @ bv.T, np.abs(av) @ np.abs(bv).T, 128 * n, "wgrad of group %d" % e)
        at += 128 * n


@pytest.mark.parametrize("M,N,K,plan", [(267, 3904, 2992, (256, 2)), (1229, 400, 5072, (256, 4)), (19, 4112, 3376, (32, 4))])
def test_shared_products_in_order_and_captured(M, N, K, plan):
    """Quantisation, a product of shared tiles only, and a reader of D in one chain on a stream, then the chain replayed
    from a graph over changed inputs."""
    fd, dev = _fd()
    got = fd.fp8_block_gemm_plan(M, N, K)
    _expect((got[0], got[1], got[2]), plan + (0,), dev)
    b, b_s = _dev(dev, *_operand(N, K, 0, "shared chain", 128))
    x = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    q, s = torch.empty((M, K), dtype=torch.uint8, device=dev), torch.empty((br.blocks(K), M), device=dev)
    D, out = (torch.empty((M, N), dtype=torch.bfloat16, device=dev) for _ in range(2))
    g = wl.generator(303, "shared chain")
    xs = [wl.normal((M, K), 1.0, g, torch.bfloat16).to(dev) for _ in range(3)]

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
    torch.cuda.synchronize()
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
