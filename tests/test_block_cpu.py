"""Block-scaled FP8 without a GPU: sizes, and the refusals of the C entries and of the binding
(every check comes before the first launch)."""
import numpy as np
import pytest
import torch

import block_reference as br


@pytest.fixture(scope="module")
def fd():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_delayed_scaling_gb300
    return fp8_delayed_scaling_gb300


def test_padded_rows(fd):
    assert [fd.fp8_block_padded_rows(n) for n in (0, 1, 128, 129, 1000)] == [0, 128, 128, 256, 1024]
    rng = np.random.default_rng(5)
    for _ in range(300):  # the bound covers every way to cut the rows, and is met: one row each
        rows, g = int(rng.integers(1, 600)), int(rng.integers(1, 40))
        cuts = np.sort(rng.integers(0, rows + 1, g - 1))
        lens = np.diff(np.concatenate([[0], cuts, [rows]]))
        assert sum(br.blocks(n) * 128 for n in lens) <= fd.fp8_block_padded_rows(rows, g)
    assert fd.fp8_block_padded_rows(7, 7) == 7 * 128 and fd.fp8_block_padded_rows(7, 1000) == 7 * 128


def test_c_entries_refuse_on_the_host(fd):
    L, a = fd._lib, 1 << 20  # a fake, 16-byte aligned address: validation fails before any use
    quant = lambda x=a, xd=1, rows=32, cols=64, off=None, g=0, fmt=0, rq=a, rs=a, cq=a, cs=a, db=None, ws=None, wb=0: (  # noqa: E731
        L.fp8_block_quantize(x, xd, rows, cols, off, g, fmt, rq, rs, cq, cs, db, ws, wb, None))
    assert quant(x=None) == fd.ERR_INVALID_ARG
    assert quant(xd=2) == fd.ERR_INVALID_ARG
    assert quant(fmt=2) == fd.ERR_INVALID_ARG
    assert quant(rows=-1) == fd.ERR_SHAPE
    assert quant(rows=1 << 31) == fd.ERR_SHAPE
    assert quant(cols=0) == fd.ERR_SHAPE
    assert quant(cols=24) == fd.ERR_SHAPE
    assert quant(g=3) == fd.ERR_INVALID_ARG            # groups without offsets
    assert quant(off=a, g=0) == fd.ERR_INVALID_ARG
    assert quant(off=a, g=1025) == fd.ERR_INVALID_ARG
    assert quant(off=a + 2, g=4) == fd.ERR_ALIGN
    assert quant(off=a, g=4, db=a, ws=a, wb=1 << 20) == fd.ERR_INVALID_ARG  # no bias gradient per group
    assert quant(rq=None, rs=None, cq=None, cs=None) == fd.ERR_INVALID_ARG
    assert quant(rs=None) == fd.ERR_INVALID_ARG        # codes without their factors
    assert quant(cq=None) == fd.ERR_INVALID_ARG
    assert quant(x=a + 8) == fd.ERR_ALIGN
    assert quant(cs=a + 4) == fd.ERR_ALIGN
    assert quant(db=a) == fd.ERR_WORKSPACE
    assert quant(db=a, ws=a, wb=fd.fp8_cast_workspace_size(32, 64) - 1) == fd.ERR_WORKSPACE
    weight = lambda w=a, n=1, rows=32, cols=64, q=a, s=a, qt=a, st=a, fmt=0: L.fp8_block_quantize_weight(  # noqa: E731
        w, 1, n, rows, cols, fmt, q, s, qt, st, None)
    assert weight(w=None) == fd.ERR_INVALID_ARG
    assert weight(n=0) == fd.ERR_INVALID_ARG
    assert weight(n=65536) == fd.ERR_INVALID_ARG
    assert weight(rows=0) == fd.ERR_SHAPE
    assert weight(cols=40) == fd.ERR_SHAPE
    assert weight(s=None) == fd.ERR_INVALID_ARG
    assert weight(q=None, s=None, qt=None, st=None) == fd.ERR_INVALID_ARG
    assert weight(qt=a + 8) == fd.ERR_ALIGN
    gemm = lambda A=a, ad=0, bs=a, per=128, M=32, N=64, K=64, bias=None, bd=1, D=a, dd=1: L.fp8_block_gemm(  # noqa: E731
        A, ad, a, a, 0, bs, per, M, N, K, bias, bd, D, dd, None, None)
    assert gemm(A=None) == fd.ERR_INVALID_ARG
    assert gemm(ad=2) == fd.ERR_INVALID_ARG
    assert gemm(dd=2) == fd.ERR_INVALID_ARG
    assert gemm(per=64) == fd.ERR_INVALID_ARG
    assert gemm(bias=a, bd=3) == fd.ERR_INVALID_ARG
    assert gemm(M=-1) == fd.ERR_SHAPE
    assert gemm(N=8) == fd.ERR_SHAPE
    assert gemm(K=0) == fd.ERR_SHAPE
    assert gemm(K=72) == fd.ERR_SHAPE
    assert gemm(bs=a + 8) == fd.ERR_ALIGN
    assert gemm(bias=a + 8) == fd.ERR_ALIGN
    grouped = lambda off=a, g=4, M=32, N=64, K=64, D=a: L.fp8_block_gemm_grouped(  # noqa: E731
        a, 0, a, a, 0, a, off, g, M, N, K, D, 1, None, None)
    assert grouped(off=None) == fd.ERR_INVALID_ARG
    assert grouped(g=0) == fd.ERR_INVALID_ARG
    assert grouped(g=1025) == fd.ERR_INVALID_ARG
    assert grouped(off=a + 1) == fd.ERR_ALIGN
    assert grouped(D=None) == fd.ERR_INVALID_ARG
    assert grouped(N=24) == fd.ERR_SHAPE
    assert grouped(g=1024, N=1 << 22) == fd.ERR_SHAPE  # B has 2^32 rows
    wgrad = lambda off=a, g=4, M=48, N=64, T=256, A=a, D=a: L.fp8_block_gemm_grouped_wgrad(  # noqa: E731
        A, 1, a, a, 0, a, off, g, M, N, T, D, 1, None, None)
    assert wgrad(T=200) == fd.ERR_SHAPE
    assert wgrad(M=0) == fd.ERR_SHAPE
    assert wgrad(g=1024, M=1 << 22) == fd.ERR_SHAPE    # D has 2^32 rows
    assert wgrad(N=8) == fd.ERR_SHAPE
    assert wgrad(A=None) == fd.ERR_INVALID_ARG
    assert wgrad(D=None, T=0) == fd.ERR_INVALID_ARG
    assert wgrad(off=None) == fd.ERR_INVALID_ARG
    assert fd.fp8dl_last_error() != ""


def test_binding_refuses_shapes_types_strides_and_cpu_tensors(fd):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    f32 = lambda *s: torch.zeros(s)  # noqa: E731
    x = torch.zeros((40, 272), dtype=torch.bfloat16)
    ok = dict(row_q=u8(40, 272), row_s=f32(3, 40), col_q=u8(272, 128), col_s=f32(1, 272))
    bad = [dict(ok, row_q=u8(40, 256)), dict(ok, row_s=f32(40, 3)), dict(ok, col_q=u8(272, 40)),
           dict(ok, col_s=f32(2, 272)), dict(ok, row_q=u8(272, 40).t()), dict(ok, row_s=f32(3, 40).double()),
           dict(ok, offsets=torch.zeros(3)), dict(ok, offsets=torch.zeros(1, dtype=torch.int32)), ok]
    for kw in bad:  # the last one is well-formed, but on the CPU
        with pytest.raises(ValueError):
            fd.fp8_block_quantize(x, fd.E4M3, **kw)
    with pytest.raises(ValueError):
        fd.fp8_block_quantize(x.t(), fd.E4M3, **ok)
    with pytest.raises(TypeError):
        fd.fp8_block_quantize(x.half(), fd.E4M3, **ok)
    w = torch.zeros((2, 144, 272))
    with pytest.raises(ValueError):
        fd.fp8_block_quantize_weight(w, fd.E4M3, q=u8(2, 144, 272), s=f32(2, 2, 3))
    A, As, B, Bs, D = u8(5, 256), f32(2, 5), u8(144, 256), f32(2, 2), f32(5, 144)
    for args in ((A, As.t(), B, Bs, D), (A, As, B, f32(2, 3), D), (A, As, B, Bs, f32(144, 5)), (A, As, u8(144, 128), Bs, D),
                 (A, As, B, Bs, D), (A[:, ::2], As, B[:, ::2], Bs, D)):
        with pytest.raises(ValueError):
            fd.fp8_block_gemm(args[0], 0, args[1], args[2], 0, args[3], args[4])
    with pytest.raises(ValueError):
        fd.fp8_block_gemm(A, 0, As, B, 0, Bs, D, bias=f32(5))
    off = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):  # offsets for three groups, two weights
        fd.fp8_block_gemm_grouped(A, 0, As, u8(2, 144, 256), 0, f32(2, 2, 2), off, D)
    with pytest.raises(ValueError):  # the factors of the transposed copy
        fd.fp8_block_gemm_grouped(A, 0, As, u8(3, 144, 256), 0, f32(3, 3, 2), off, D)
    with pytest.raises(ValueError):
        fd.fp8_block_gemm_grouped_wgrad(u8(48, 256), 1, f32(2, 48), u8(64, 128), 0, f32(1, 64), off, f32(3, 48, 64))


def test_layers_refuse_before_any_launch(fd):
    from fp8_delayed_scaling_gb300.blocklinear import BlockExperts, BlockLinear
    lin = BlockLinear(torch.zeros((32, 16), dtype=torch.bfloat16), None, 8)
    with pytest.raises(RuntimeError):
        lin.forward(torch.zeros((8, 16), dtype=torch.bfloat16), is_first_microbatch=False)
    with pytest.raises(RuntimeError):
        lin.backward(torch.zeros((8, 32), dtype=torch.bfloat16))
    ex = BlockExperts(torch.zeros((3, 32, 16), dtype=torch.bfloat16), 8)
    with pytest.raises(RuntimeError):
        ex.backward(torch.zeros((8, 32), dtype=torch.bfloat16))
    with pytest.raises(ValueError):  # more rows than the layer was made for
        ex.x8.quantize(torch.zeros((9, 16), dtype=torch.bfloat16), 0)


def test_reference_quantiser_by_hand():
    """The plain quantiser the GPU tests compare with, on blocks whose scale is worked out by hand."""
    x = np.zeros((2, 130), np.float32)
    x[0, 0], x[0, 1] = 7.0, -1.0      # scale 448 / 7 = 64
    x[0, 129] = 3.5                   # a block of two: scale 128
    q, s = br.rows(x, 0)
    v = torch.from_numpy(q).view(torch.float8_e4m3fn).float().numpy()
    assert v[0, 0] == 448 and v[0, 1] == -64 and v[0, 129] == 448
    assert s[0, 0] == np.float32(1 / 64) and s[1, 0] == np.float32(1 / 128) and s[0, 1] == 1.0
    assert np.array_equal(br.values(q, 0, s, 1), x.astype(np.float64))
    t, ts, used = br.cols(x.T.copy(), 0, [0, 1, 1, 130])
    assert used == 128 + 256 and t.shape == (2, 384)  # 1, 0 and 129 rows
    assert ts.shape == (3, 2)
