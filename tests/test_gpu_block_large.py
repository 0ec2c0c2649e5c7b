"""Block-scaled FP8 past 2^31 bytes or elements of an operand or a result: every offset is a 64-bit one.  Inputs are
drawn on the GPU; sampled rows and columns, those around the border among them, are computed again in fp64."""
import numpy as np
import pytest
import torch

import block_reference as br
from helpers import gpu

pytestmark = pytest.mark.gpu

EDGE = 1 << 31


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _fd():
    import fp8_delayed_scaling_gb300 as fd
    return fd, gpu()


def _near(n, ld):
    """Rows of [n x ld] to look at: the first and last, those around element 2^31, some between."""
    e = EDGE // ld
    rows = [0, 1, 127, 128, n // 3, e - 1, e, e + 1, n - 129, n - 2, n - 1]
    return torch.tensor(sorted({r for r in rows if 0 <= r < n}))


def _random_codes(shape, g, fmt, dev):
    """E4M3 or E5M2 codes without NaN and infinities."""
    q = torch.randint(0, 256, shape, dtype=torch.uint8, device=dev, generator=g)
    mag = q & 0x7F
    bad = (mag == 0x7F) if fmt == 0 else (mag >= 0x7C)
    return q.masked_fill_(bad, 0x38)


def _factors(shape, g, dev):
    return torch.rand(shape, device=dev, generator=g) + 0.5


def _decoded(q, fmt, s):
    """fp64 values of a few rows' codes q [r x K] with their factors s [K/128 x r]."""
    return q.view(br.F8[fmt]).double() * s.double().t().repeat_interleave(128, 1)[:, :q.shape[1]]


def _check(got, a, b, K, what):
    br.check(got, (a @ b.t()).cpu().numpy(), (a.abs() @ b.abs().t()).cpu().numpy(), K, what)


@pytest.mark.parametrize("groups", [False, True])
def test_quantize(groups):
    fd, dev = _fd()
    R, C = 65536 + 40, 40960
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.empty((R, C), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    off = [0, 1, 700, 700, 52000, 52429, 65500] if groups else None
    G = len(off) - 1 if groups else 0
    T = fd.fp8_block_padded_rows(R, G)
    row_q, col_q = torch.zeros((R, C), dtype=torch.uint8, device=dev), torch.zeros((C, T), dtype=torch.uint8, device=dev)
    row_s, col_s = torch.zeros((C // 128, R), device=dev), torch.zeros((T // 128, C), device=dev)
    fd.fp8_block_quantize(x, fd.E4M3, row_q=row_q, row_s=row_s, col_q=col_q, col_s=col_s,
                          offsets=torch.tensor(off, dtype=torch.int32, device=dev) if groups else None)
    rows = _near(off[-1] if groups else R, C)
    q, s = br.rows(x[rows.to(dev)].float().cpu().numpy(), 0)
    assert np.array_equal(row_q[rows.to(dev)].cpu().numpy(), q)
    assert np.array_equal(row_s[:, rows.to(dev)].cpu().numpy(), s)
    cols = _near(C, T)
    qt, st, used = br.cols(x[:, cols.to(dev)].float().cpu().numpy(), 0, off)
    assert np.array_equal(col_q[cols.to(dev), :used].cpu().numpy(), qt[:, :used])
    assert np.array_equal(col_s[:used // 128, cols.to(dev)].cpu().numpy(), st[:used // 128])
    if groups:
        assert torch.all(row_q[off[-1]:] == 0) and torch.all(col_q[:, used:] == 0)


def test_quantize_weight():
    fd, dev = _fd()
    E, R, C = 20, 8208, 16400
    g = torch.Generator(device=dev).manual_seed(2)
    w = torch.empty((E, R, C), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    q, q_t = torch.zeros((E, R, C), dtype=torch.uint8, device=dev), torch.zeros((E, C, R), dtype=torch.uint8, device=dev)
    s, s_t = torch.zeros((E, br.blocks(C), br.blocks(R)), device=dev), torch.zeros((E, br.blocks(R), br.blocks(C)), device=dev)
    fd.fp8_block_quantize_weight(w, fd.E4M3, q=q, s=s, q_t=q_t, s_t=s_t)
    for e in (0, EDGE // (R * C), E - 1):
        for i in (0, R // 128 - 1, R // 128):  # blocks of rows, the last one short
            part = w[e, 128 * i:128 * i + 128].float().cpu().numpy()
            rq, rs = br.weight(part, 0)
            assert np.array_equal(q[e, 128 * i:128 * i + 128].cpu().numpy(), rq)
            assert np.array_equal(q_t[e, :, 128 * i:128 * i + 128].cpu().numpy(), rq.T)
            assert np.array_equal(s[e, :, i].cpu().numpy(), rs[:, 0]) and np.array_equal(s_t[e, i].cpu().numpy(), rs[:, 0])


@pytest.mark.parametrize("M,N,K", [(65536 + 8, 40960, 144),   # D
                                   (65536 + 8, 400, 40960),   # A
                                   (7, 65536 + 16, 40960),    # B, few rows
                                   (300, 65536 + 16, 40960)])  # B, many
def test_product(M, N, K):
    fd, dev = _fd()
    g = torch.Generator(device=dev).manual_seed(3)
    a, b = _random_codes((M, K), g, 0, dev), _random_codes((N, K), g, 1, dev)
    a_s, b_s = _factors((br.blocks(K), M), g, dev), _factors((br.blocks(K), br.blocks(N)), g, dev)
    D = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=dev)
    fd.fp8_block_gemm(a, 0, a_s, b, 1, b_s, D)
    ms, ns = _near(M, max(N, K)).to(dev), _near(N, K).to(dev)
    if M * N > EDGE:  # whole rows of D
        ns = torch.arange(N, device=dev)
    _check(D[ms][:, ns], _decoded(a[ms], 0, a_s[:, ms]), _decoded(b[ns], 1, b_s[:, ns // 128]), K, "product")


@pytest.mark.parametrize("M", [300, 6000])  # few rows a group, and many
def test_grouped_weights(M):
    fd, dev = _fd()
    G, N, K = 17, 8208, 20480
    g = torch.Generator(device=dev).manual_seed(4)
    a, b = _random_codes((M, K), g, 0, dev), _random_codes((G, N, K), g, 0, dev)
    a_s, b_s = _factors((br.blocks(K), M), g, dev), _factors((G, br.blocks(K), br.blocks(N)), g, dev)
    off = [M * e // G for e in range(G + 1)]
    D = torch.full((M, N), 7.0, device=dev)
    fd.fp8_block_gemm_grouped(a, 0, a_s, b, 0, b_s, torch.tensor(off, dtype=torch.int32, device=dev), D)
    ns = torch.tensor([0, 1, 127, 128, 5000, N - 17, N - 1], device=dev)
    for e in (0, EDGE // (N * K), EDGE // (N * K) + 1, G - 1):
        ms = torch.tensor(sorted({off[e], off[e] + 1, (off[e] + off[e + 1]) // 2, off[e + 1] - 1}), device=dev)
        _check(D[ms][:, ns], _decoded(a[ms], 0, a_s[:, ms]), _decoded(b[e, ns], 0, b_s[e][:, ns // 128]), K, "group %d" % e)


@pytest.mark.parametrize("M,N,G,T", [(10256, 48, 3, 1 << 18),   # A: the transposed codes
                                     (8200, 8208, 40, 40 * 128)])  # D: all groups' gradients
def test_grouped_wgrad(M, N, G, T):
    fd, dev = _fd()
    g = torch.Generator(device=dev).manual_seed(5)
    a, b = _random_codes((M, T), g, 1, dev), _random_codes((N, T), g, 0, dev)
    a_s, b_s = _factors((T // 128, M), g, dev), _factors((T // 128, N), g, dev)
    off = [T // 128 * e // G * 128 for e in range(G + 1)]  # whole blocks: the padded length is the rows'
    D = torch.full((G, M, N), 7.0, dtype=torch.bfloat16, device=dev)
    fd.fp8_block_gemm_grouped_wgrad(a, 1, a_s, b, 0, b_s, torch.tensor(off, dtype=torch.int32, device=dev), D)
    ms, ns = _near(M, T).to(dev), torch.tensor([0, 1, 15, N // 2, N - 2, N - 1], device=dev)
    for e in sorted({0, 1, EDGE // (M * N) if EDGE // (M * N) < G else 0, G - 1}):
        k = slice(off[e], off[e + 1])
        kb = slice(off[e] // 128, off[e + 1] // 128)
        _check(D[e][ms][:, ns], _decoded(a[ms, k], 1, a_s[kb][:, ms]), _decoded(b[ns, k], 0, b_s[kb][:, ns]),
               off[e + 1] - off[e], "group %d" % e)
