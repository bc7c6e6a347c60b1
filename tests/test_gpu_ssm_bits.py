"""How many bits the tensor-core scan keeps where the bounds of test_gpu_ssm.py leave it room.

Outputs.  In sequences of 17 to 128 tokens that start from zero no copy of the
state is read, so an output's only roundings to bf16 are its own (half a step)
and the decayed scores', which are two bf16 terms: what is left of a score is at
most 2^-8 of what is left after the first term, itself at most 2^-8 of the score,
so 2^-16 of each term of the sum.  The fp32 part is the other test's.

States.  The state's updates are three bf16 terms, so at most 2^-24 of an update is
left; two would leave up to 2^-16, 256 times as much.  x is not 0 at a few tokens
only, so an entry of the state is a sum of that many products B (d x): d, d x and its
split cost 3 2^-24 of each, the three terms' sum, each product's way into the state and
their sum 2 2^-24 and one for each term, and the products themselves are exact.  With a
decay, the exponent is a sum of l that is off by at most 40 2^-24 of its length L, the
exponentials by 2^-22 for the token and for each chunk that the term passes."""
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
    return y.double().cpu().numpy(), None if st is None else st.double().cpu().numpy()  # (no ctx: the pool is only written)


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


def _sparse(T, at, A, N, P, seed):
    """Inputs whose x is 0 but at the tokens `at`, with steps that fill 24 bits; small ones in between."""
    v = _inputs(T, 2, 1, N, P, BF, seed, 1)
    keep = torch.zeros(T, dtype=torch.bool)
    keep[at] = True
    v["x"][~keep] = 0
    v["A"] = torch.tensor(A)
    v["dt"] = (v["dt"].float().abs() * 0.004).to(BF)
    v["dt"][keep] = (0.25 + 0.5 * torch.rand(len(at), 2, generator=torch.Generator().manual_seed(seed))).to(BF)
    v["dt_bias"] = torch.tensor([0.001234567, 0.0009876543])
    return v


def _states_with_terms(n, terms, at):
    """The final state (no decay) with d x in that many bf16 terms: what a kernel with fewer would leave."""
    S = np.zeros((1, 2, n["B"].shape[2], n["x"].shape[2]))
    for t in at:
        d = np.float32(n["dt"][t] + n["dt_bias"])
        v, kept = torch.from_numpy((d[:, None] * np.float32(n["x"][t])).astype(np.float32)), 0
        for _ in range(terms):
            q = v.to(BF).float()
            kept, v = kept + q.double(), v - q
        S[0] += n["B"][t, 0][None, :, None] * kept.numpy()[:, None, :]
    return S


@pytest.mark.parametrize("N,P", [(16, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("A", [[0.0, 0.0], [-0.25, -1.0]])
@pytest.mark.parametrize("T,at", [(100, [57]), (200, [3, 150]), (3000, [70, 1500, 2990])])
def test_states_keep_24_bits(T, at, A, N, P):
    v = _sparse(T, at, A, N, P, T + N)
    _, st = _scan(v, softplus=False)
    n = {k: _n(t) for k, t in v.items()}
    n["state"] = np.zeros_like(n["state"])
    _, ref, _ = serving.ssm_scan(**n, R=1, softplus=False)
    d = n["dt"] + n["dt_bias"]
    u, tol = 2.0 ** -24, np.zeros_like(ref)
    for t in at:
        L = -(d[t + 1:] * n["A"]).sum(0)  # the term's way to the end
        term = np.abs(n["B"][t, 0][None, :, None] * (d[t][:, None] * n["x"][t])[:, None, :]) * np.exp(-L)[:, None, None]
        decay = 0 if not n["A"].any() else 4 * (2 + (T - t) // 128) + 40 * L[:, None, None]
        tol[0] += (5 + len(at) + decay) * u * term
    off = lambda s: np.abs(s - ref) / np.maximum(tol, 1e-300)
    assert (off(st) <= 1).all(), float(np.nanmax(off(st)))
    if not n["A"].any():  # the bound tells two terms from three
        assert off(_states_with_terms(n, 3, at)).max() <= 1 and off(_states_with_terms(n, 2, at)).max() > 8
