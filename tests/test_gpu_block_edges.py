"""Block-scaled FP8 where its arithmetic reaches an end: overlapping groups of more than 2^32 blocks."""
import pytest
import torch

import block_reference as br
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
