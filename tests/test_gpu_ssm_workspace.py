"""kda_ssm_scan stays inside the workspace that kda_ssm_scan_workspace_size asks for: guard
words behind it are never written, for sequences cut anywhere and contexts that begin
anywhere in a chunk."""
import numpy as np
import pytest
import torch

from gated_delta_rule_117_b200 import kda

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
GUARD, FILL = 1 << 20, 0x7FC12345  # words; a NaN that no sum leaves behind


def _cuts(g, R, rows):
    """Offsets of R sequences over all the rows: even, random, one long, all but one empty."""
    kind = g.integers(4)
    if kind == 0:
        c = np.arange(1, R) * rows // R
    elif kind == 1:
        c = np.sort(g.integers(0, rows + 1, R - 1))
    elif kind == 2:
        c = np.arange(1, R) if g.random() < 0.5 else rows - np.arange(R - 1, 0, -1)
    else:
        c = np.where(np.arange(1, R) <= g.integers(R), 0, rows)
    return np.concatenate([[0], c, [rows]]).astype(np.int32)


# segments of 16 to 128 tokens on the CUDA cores, of 512 and more on the tensor cores
@pytest.mark.parametrize("dtype,R,rows,H,N,P", [(F32, 1, 300, 2, 16, 16), (F32, 2, 700, 2, 64, 32), (F32, 5, 1500, 1, 16, 32), (F32, 1, 4099, 2, 32, 32),
                                               (F32, 12, 900, 2, 16, 16), (BF, 1, 3000, 1, 64, 64), (BF, 3, 6001, 2, 16, 128),
                                               (BF, 2, 9000, 1, 128, 64), (BF, 1, 300, 2, 16, 17)])
def test_guard_words(dtype, R, rows, H, N, P):
    misaligned = P == 17  # (bf16 rows that only the CUDA-core kernel takes)
    P = 16 if misaligned else P
    g = np.random.default_rng(rows)
    code = kda.KDA_DTYPE_BF16 if dtype is BF else kda.KDA_DTYPE_F32
    need = kda.kda_ssm_scan_workspace_size(R, rows, H, 1, N, P, code)
    assert 0 < need and need % 16 == 0
    rn = lambda *s: torch.randn(*s, device="cuda").to(dtype)
    x = rn(rows, H * P + 1)[:, 1:].unflatten(1, (H, P)) if misaligned else rn(rows, H, P)
    dt, B, C, A = rn(rows, H), rn(rows, 1, N), rn(rows, 1, N), -torch.ones(H, device="cuda")
    ws = torch.empty(need // 4 + GUARD, dtype=torch.int32, device="cuda")
    pool, bias = torch.zeros(R, H, N, P, device="cuda"), torch.full((H,), -4.0, device="cuda")
    segmented = 0
    for k in range(40):
        packed = R > 1 and k % 4 > 0
        if not packed and rows % R:
            continue
        ws.fill_(FILL)
        ctx = torch.from_numpy(g.integers(0, 300, R).astype(np.int32)).cuda()
        cu = torch.from_numpy(_cuts(g, R, rows)).cuda() if packed else None
        args = [t if packed or R == 1 else t.unflatten(0, (R, -1)) for t in (x, dt, B, C)]
        y = kda.ssm_scan(args[0], args[1], A, args[2], args[3], dt_bias=bias, state=pool, ctx=ctx, cu=cu, workspace=ws.view(torch.uint8)[:need])
        assert torch.isfinite(y.float()).all() and (ws[need // 4:] == FILL).all()
        segmented += int((ws[:need // 4] != FILL).any())
    assert segmented > 0 and kda.kda_get_device_status() == 0
