"""How many bits the tensor-core scan keeps where the bounds of test_gpu_ssm.py leave it room.

Outputs.  In sequences of 17 to 128 tokens that start from zero no copy of the
state is read, so an output's only roundings to bf16 are its own (half a step)
and the decayed scores', which are two bf16 terms: what is left of a score is at
most 2^-8 of what is left after the first term, itself at most 2^-8 of the score,
so 2^-16 of each term of the sum.  The fp32 part is the other test's."""
import numpy as np
import pytest
import torch

from gated_delta_rule_117_b200 import kda
from oracle import serving
from test_gpu_ssm import _inputs, _n

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _scan(v, **kw):
    d = {k: None if t is None else t.cuda() for k, t in v.items()}
    st = d.pop("state")
    y = kda.ssm_scan(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["dt_bias"], state=st, **kw)
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == 0
    return y.double().cpu().numpy(), None if st is None else st.double().cpu().numpy()


@pytest.mark.parametrize("N,P", [(16, 64), (64, 16), (128, 64), (128, 128)])
@pytest.mark.parametrize("slow", [1.0, 0.05])
@pytest.mark.parametrize("lens", [[128, 100, 17, 77, 127], [33], [128]])
def test_outputs_of_one_chunk(lens, slow, N, P):
    rows, R, H, T = sum(lens), len(lens), 4, max(lens)
    v = _inputs(rows, H, 2, N, P, BF, N + P + rows, 1, slow)
    v["state"] = None
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    y, _ = _scan(v, cu=torch.from_numpy(cu).cuda())
    n = {k: _n(t) for k, t in v.items()}
    ref, _, _ = serving.ssm_scan(**n, cu=cu, R=R)
    a = {k: np.abs(t) if t is not None and k in ("x", "B", "C", "D") else t for k, t in n.items()}
    yabs, _, _ = serving.ssm_scan(**a, cu=cu, R=R)
    a["A"] = a["A"] / 2
    yslow, _, _ = serving.ssm_scan(**a, cu=cu, R=R)
    u = 2.0 ** -24
    e = ((3 * T + N + 16) * u + 2.0 ** -16) * yabs + 10 * u * yslow
    tol = e + torch.finfo(BF).eps / 2 * (np.abs(ref) + e)
    off = np.abs(y - ref) / tol
    assert (off <= 1).all(), float(np.nanmax(off))
