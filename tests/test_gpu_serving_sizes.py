"""Sizes beyond 32 bits are refused by the Python helpers, not cut to their low bits."""
import pytest
import torch

from gated_delta_rule_117_b200 import kda

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
FAR = 1 << 32


def test_numbers():
    i32 = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for page, rows in ((FAR + 16, 8), (16, FAR + 8)):
        with pytest.raises(ValueError, match="2\\^31"):
            kda.block_map(i32, None, i32, table, page, rows)
    x, w = torch.zeros(4, 32, device="cuda"), torch.zeros(32, 4, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        kda.short_conv(x, w, head_dim=FAR + 16, l2norm=True)
    with pytest.raises(ValueError, match="2\\^31"):
        kda.short_conv_step(x, w, torch.zeros(4, 3, 32, device="cuda"), head_dim=FAR + 16, l2norm=True)
    s, a = torch.zeros(300, 1, 16, device="cuda"), torch.zeros(1, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        kda.ssm_scan(s, s[:, :, 0], a, s, s, block_table=table[:1], pages=torch.zeros(1, 1, 16, 16, device="cuda"), page_size=FAR + 128)


def test_rows_and_pool_entries():
    far = torch.empty(FAR + 5, 1, dtype=BF, device="cuda")  # 8.6 GB, never read
    w = torch.zeros(1, 2, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        kda.short_conv(far, w)
    with pytest.raises(ValueError, match="2\\^31"):
        kda.short_conv(far[:5], w, state=far[:, None])
    with pytest.raises(ValueError, match="2\\^31"):
        kda.short_conv_step(far[:5], w, far[:, None])
