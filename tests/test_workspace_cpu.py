"""A workspace that has fewer bytes than its shape says (an expanded or strided view) is refused before anything is launched."""
import pytest
import torch


@pytest.fixture(scope="module")
def fd():
    import __graft_entry__ as g
    g.build()
    import fp8_delayed_scaling_gb300 as fd
    return fd


VIEWS = [lambda: torch.zeros(1, dtype=torch.uint8).expand(1 << 20), lambda: torch.zeros(1 << 12, dtype=torch.uint8)[::4]]


@pytest.mark.parametrize("view", VIEWS)
def test_views_are_no_workspaces(fd, view):
    i32, f32, u8 = (lambda *s, d=d: torch.zeros(s, dtype=d) for d in (torch.int32, torch.float32, torch.uint8))
    T, E, k = 6, 10, 3
    refuses = lambda: pytest.raises(ValueError, match="workspace must be contiguous")  # noqa: E731
    with refuses():
        fd.moe_route(f32(T, E), i32(T, k), f32(T, k), i32(T, k), i32(T * k), i32(E + 1), workspace=view())
    with refuses():
        fd.fp8_block_dact(f32(5, 144), u8(5, 144), 0, f32(2, 5), fd.ACT_SILU, 0, dbias=f32(144), workspace=view())
    with refuses():
        fd.fp8_block_quantize(f32(5, 144), 0, row_q=u8(5, 144), row_s=f32(2, 5), dbias=f32(144), workspace=view())
