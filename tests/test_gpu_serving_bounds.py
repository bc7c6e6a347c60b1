"""Offsets that lead outside the rows are recorded, wherever the sequence that they
cut off begins, and its rows and pool entry stay as they were."""
import pytest
import torch

from gated_delta_rule_117_b200 import kda

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DEVICE = 10


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("C", [8, 7, 1100])
@pytest.mark.parametrize("cu,good", [([0, 6, 9], [0]), ([0, 6, 6, 4000], [0, 1]), ([6, 9], []), ([2000, 3000], []), ([-5, 3, 6], [1]),
                                     ([0, 3, 9], [0]), ([0, 4, 6], [0, 1])])
def test_convolution(cu, good, C):
    x, w = torch.randn(6, C, device="cuda"), torch.randn(C, 4, device="cuda")
    R = len(cu) - 1
    pool, y = torch.full((R, 3, C), 5.0, device="cuda"), torch.full((6, C), 7.0, device="cuda")
    kda.short_conv(x, w, state=pool, cu=_i32(cu), y=y)
    assert kda.kda_get_device_status() == (0 if len(good) == R else DEVICE)
    seen = torch.zeros(6, dtype=torch.bool)
    for r in range(R):
        empty = cu[r] == cu[r + 1]
        assert ((pool[r] == 5.0).all() or not (r not in good or empty)) and (r not in good or empty or (pool[r] != 5.0).any())
        if r in good:
            seen[cu[r]:cu[r + 1]] = True
            assert torch.equal(y[cu[r]:cu[r + 1]], kda.short_conv(x[cu[r]:cu[r + 1]], w))
    assert (y[(~seen).cuda()] == 7.0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows", [40, 2100])  # whole sequences, and segments
@pytest.mark.parametrize("cu,good", [([0, 1, 1.5], [0]), ([1, 2], []), ([9, 12], []), ([0, 0.5, 1, 1, 90], [0, 1, 2]), ([-0.5, 0.5, 1], [1])])
def test_scan(cu, good, rows, dtype):
    cu = [int(c * rows) for c in cu]
    H, N, P, R = 2, 32, 64, len(cu) - 1
    rn = lambda *s: torch.randn(*s, device="cuda").to(dtype)
    x, dt, B, C = rn(rows, H, P), rn(rows, H), rn(rows, 1, N), rn(rows, 1, N)
    A = torch.tensor([-1.0, -3.0], device="cuda")
    pool, y = torch.full((R, H, N, P), 5.0, device="cuda"), torch.full_like(x, 7.0)
    kda.ssm_scan(x, dt, A, B, C, state=pool, cu=_i32(cu), y=y)
    assert kda.kda_get_device_status() == DEVICE
    seen = torch.zeros(rows, dtype=torch.bool)
    for r in range(R):
        if r not in good or cu[r] == cu[r + 1]:
            assert (pool[r] == 5.0).all()
        else:
            assert (pool[r] != 5.0).any() and torch.isfinite(y[cu[r]:cu[r + 1]].float()).all()
            seen[cu[r]:cu[r + 1]] = True
    assert (y[(~seen).cuda()] == 7.0).all() and (y[seen.cuda()] != 7.0).any() == bool(seen.any())
