"""Steps that wipe the state out in the middle of a sequence (kda_ssm_scan asks
only for d >= 0 and A <= 0): the tokens behind such a step see each other
through their own small decays, whatever the step was.

x is 0 at those tokens, so that their own contribution (d times larger than the
others') does not hide the rest.  The tolerance is the one derived in
test_gpu_ssm.py: a term that crosses a wiping step is 0 in fp32 and in 64 bits
alike, so only terms whose decays it bounds are left."""
import numpy as np
import pytest
import torch

from gated_delta_rule_117_b200 import kda
from oracle import serving
from test_gpu_ssm import _inputs, _n, _tolerances

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _check(T, step, at, dtype, A=None, small=None, N=32, P=64):
    H = 2
    v = _inputs(T, H, 1, N, P, dtype, T + len(at), 1)
    if A is not None:
        v["A"] = torch.tensor(A)
    if small is not None:
        v["dt_bias"] = torch.full((H,), float(np.log(np.expm1(small))))
    for t in at:
        v["dt"][t] = step
        v["x"][t] = 0
    d = {k: t.cuda() for k, t in v.items()}
    pages, table = torch.full((T // 128 + 1, H, N, P), 3.0), np.arange(T // 128, dtype=np.int32)[None] + 1
    st, pg = d.pop("state"), pages.cuda()
    y = kda.ssm_scan(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["dt_bias"], state=st, ctx=torch.zeros(1, dtype=torch.int32, device="cuda"),
                     block_table=torch.from_numpy(table).cuda(), pages=pg, page_size=128)
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == 0
    n = {k: _n(t) for k, t in v.items()}
    kw = dict(ctx=np.zeros(1), R=1, table=table, pages=_n(pages), page=128)
    ry, rs, rp = serving.ssm_scan(**n, **kw)
    for got, ref, tol in zip((y, st, pg), (ry, rs, rp), _tolerances(n, kw, T, N, dtype, ry, rs, rp)):
        off = np.abs(got.double().cpu().numpy() - ref) / np.maximum(tol, 1e-300)  # NaN fails
        assert (off <= 1).all(), float(np.nanmax(off))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("step", [1e3, 1e4, 1e5, 1e8, 1e30])
@pytest.mark.parametrize("T,at", [(40, [10]), (300, [5, 40, 47, 48, 130, 200, 255, 256]), (1500, [64, 700, 1040, 1300])])
def test_tokens_behind_a_wiping_step(T, at, step, dtype):
    _check(T, step, at, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_log_decay_beyond_fp32(dtype):
    # d A = -1e39 is -inf in fp32: a decay of 0, not of NaN (d and its products stay below 3e38)
    _check(200, 1e36, [17, 90, 140], dtype, A=[-1.0, -1000.0], small=1e-3)
