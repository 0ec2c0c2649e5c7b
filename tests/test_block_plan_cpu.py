"""fp8_block_gemm_plan without a GPU: its refusals."""
import pytest
import torch


@pytest.fixture(scope="module")
def fd():
    import __graft_entry__
    __graft_entry__.build()
    import fp8_delayed_scaling_gb300
    return fp8_delayed_scaling_gb300


def test_plan_refuses_what_the_products_refuse(fd):
    import ctypes
    out = [ctypes.byref(t()) for t in (ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64)]
    plan = lambda per=128, g=0, M=5, N=64, K=64, o=out: fd._lib.fp8_block_gemm_plan(per, g, M, N, K, *o)  # noqa: E731
    assert plan(M=0) == fd.ERR_SHAPE
    assert plan(M=1 << 31) == fd.ERR_SHAPE
    assert plan(N=24) == fd.ERR_SHAPE
    assert plan(N=1 << 29) == fd.ERR_SHAPE
    assert plan(K=72) == fd.ERR_SHAPE
    assert plan(per=64) == fd.ERR_INVALID_ARG
    assert plan(per=1, g=2) == fd.ERR_INVALID_ARG  # groups take weights
    assert plan(g=-1) == fd.ERR_INVALID_ARG
    assert plan(g=1025) == fd.ERR_INVALID_ARG
    for i in range(4):
        assert plan(o=out[:i] + [None] + out[i + 1:]) == fd.ERR_INVALID_ARG
    if not torch.cuda.is_available():
        with pytest.raises(fd.FP8DLError):
            fd.fp8_block_gemm_plan(5, 64, 64)
