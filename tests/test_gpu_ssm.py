"""Selective state space scan and step (kda_ssm_scan, kda_ssm_step) against the
fp64 oracle, element by element.

Tolerance.  Run on absolute values (|x|, |B|, |C|, |D| and the entering state's
magnitude) the oracle gives Yabs and Sabs, the sums of the magnitudes of all the
terms of an output or of an entry of the state.  In fp32 a term that t tokens
old reaches a sum through at most t decays.  The step d is off by 8 2^-24
(softplus, the sum with the bias), so a decay's exponent d A by 10 2^-24 |d A|
and the decay itself, where |d A| is below 16 in these tests, by
(10 |d A| + 2) 2^-24 of its value: summed over the term's way at most
(10 L + 3 t) 2^-24, L the sum of |d A| on it.  A term that has decayed by e^-L
is e^-L of its magnitude, and L e^-L < 1: the sum over all tokens of the first
part is covered by 10 2^-24 of the undecayed Sabs1 (the scan with A = 0 gives
it; computed with A / 2 it is tighter and still covers L e^(-L/2) < 1).  The
second part, the products and the N-term sum cost (3 T + N + 16) 2^-24 of Yabs.
The tensor-core path rounds the decayed scores, and the state that outputs
read, to bf16 (half a step, 2^-8, of each term), and splits the state's update
into bf16 pairs (2^-16).  Outputs are rounded once.  Sequences of up to 16
tokens are computed in fp32 throughout.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_117_b200 import kda
from oracle import serving

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _inputs(rows, H, G, N, P, dtype, seed, slots=1, slow=1.0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    step = torch.exp(torch.rand(H, generator=g) * 4.6 - 6.9)
    return dict(x=rn(rows, H, P).to(dtype), dt=rn(rows, H).to(dtype), B=rn(rows, G, N).to(dtype), C=rn(rows, G, N).to(dtype),
                A=-(1 + 15 * torch.rand(H, generator=g)) * slow, D=1 + 0.1 * rn(H), dt_bias=step + torch.log(-torch.expm1(-step)),
                state=0.5 * rn(slots, H, N, P))


def _n(t):
    return None if t is None else t.double().numpy() if t.is_floating_point() else t.numpy()


def _tolerances(n, kw, T, N, dtype, y, pool, pages):
    """(ytol, stol, ptol) by the rule above."""
    a = {k: np.abs(v) if v is not None and k in ("x", "B", "C", "D", "state") else v for k, v in n.items()}
    yabs, sabs, pabs = serving.ssm_scan(**a, **kw)
    a["A"] = a["A"] / 2
    yslow, sslow, pslow = serving.ssm_scan(**a, **kw)
    u = 2.0 ** -24
    lin = (3 * T + N + 16) * u
    ytol = lin * yabs + 10 * u * yslow
    slack = 0.0
    if dtype == BF:
        ytol = ytol + 2.0 ** -8 * yabs * (1 + 2.0 ** -7)
        slack = 2.0 ** -16
    half = torch.finfo(dtype).eps / 2
    ytol = ytol + half * (np.abs(y) + ytol)
    s = lambda ab, sl: None if ab is None else (lin + slack + u) * ab + 10 * u * sl
    return ytol, s(sabs, sslow), s(pabs, pslow)


def _check(lens, H, G, N, P, dtype, *, ctx=None, slots=None, packed=True, page=0, softplus=True, D=True, bias=True, seed=0,
           tail=0, state=True, slow=1.0, strided=False, n_slots=None, once=False):
    R, rows = len(lens), sum(lens)
    n_slots = (R + 2 if n_slots is None else n_slots) if state else 0
    v = _inputs(rows + tail, H, G, N, P, dtype, seed + rows + N + P, max(n_slots, 1), slow)
    if tail:
        for k in ("x", "B", "C", "dt"):
            v[k][rows:] = float("nan")
    if not state:
        v["state"] = None
    if not D:
        v["D"] = None
    if not bias:
        v["dt_bias"] = None
    if not softplus:
        v["dt"] = v["dt"].abs() * 0.05  # a step is >= 0: the call relies on it
        v["dt_bias"] = v["dt_bias"].abs() * 0.01
    i32 = lambda t: None if t is None else torch.tensor(t, dtype=torch.int32)
    cu = i32(np.concatenate([[0], np.cumsum(lens)])) if packed else None
    c, sl = i32(ctx), i32(slots)
    table = pages = None
    if page:
        cc = ctx if ctx is not None else [0] * R
        width = max((a + n) // page for a, n in zip(cc, lens)) + 1
        g = np.random.default_rng(seed)
        count = sum((a + n) // page - a // page for a, n in zip(cc, lens))
        ids, table = list(g.permutation(count + 2)), np.full((R, width), -1, np.int32)
        for r, (a, n) in enumerate(zip(cc, lens)):
            for j in range(a // page, (a + n) // page):
                table[r, j] = ids.pop()
        table = torch.from_numpy(table)
        pages = torch.full((count + 2, H, N, P), 3.0)
    dev = {k: None if t is None else t.cuda() for k, t in v.items()}
    if strided:
        xbc = torch.cat([dev["x"].flatten(1), dev["B"].flatten(1), dev["C"].flatten(1)], 1)
        dev["x"] = xbc[:, :H * P].unflatten(1, (H, P))
        dev["B"] = xbc[:, H * P:H * P + G * N].unflatten(1, (G, N))
        dev["C"] = xbc[:, H * P + G * N:].unflatten(1, (G, N))
    if not packed:
        for k in ("x", "dt", "B", "C"):
            dev[k] = dev[k].unflatten(0, (R, -1))
    st = dev.pop("state")
    y = torch.full(dev["x"].shape, 7.0, dtype=dtype, device="cuda")
    pg = None if pages is None else pages.cuda()
    dv = lambda t: None if t is None else t.cuda()
    kda.ssm_scan(dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dev["D"], dev["dt_bias"], softplus=softplus, state=st,
                 slots=dv(sl), ctx=dv(c), cu=dv(cu), block_table=dv(table), pages=pg, page_size=page, y=y)
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == 0
    n = {k: _n(t) for k, t in v.items()}
    kw = dict(softplus=softplus, slots=_n(sl), ctx=_n(c), cu=_n(cu), R=R, table=_n(table), pages=_n(pages), page=page)
    ry, rs, rp = serving.ssm_scan(**n, **kw)
    ytol, stol, ptol = _tolerances(n, kw, max(lens), N, F32 if once else dtype, ry, rs, rp)
    if once:  # sums in fp32, rounded to the type at the end
        ytol = ytol + torch.finfo(dtype).eps / 2 * (np.abs(ry) + ytol)
    yn = y.double().cpu().numpy().reshape(ry.shape)
    seen = ~np.isnan(ry[:, 0, 0])
    assert (yn[~seen] == 7.0).all()
    off = np.abs(yn - ry)[seen] / ytol[seen]
    assert (off <= 1).all(), ("y", float(off.max()))
    if st is not None:
        off = np.abs(st.double().cpu().numpy() - rs) / np.maximum(stol, 1e-300)
        assert (off <= 1).all(), ("state", float(off.max()))
    if page:
        off = np.abs(pg.double().cpu().numpy() - rp) / np.maximum(ptol, 1e-300)
        assert (off <= 1).all(), ("pages", float(off.max()))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,P", [(16, 16), (16, 128), (32, 64), (64, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens", [[1], [5, 3], [130], [64, 128, 200]])
def test_sizes(lens, N, P, dtype):
    _check(lens, 2, 1, N, P, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("H,G", [(1, 1), (6, 3), (4, 4), (3, 1)])
def test_groups(H, G, dtype):
    _check([70, 150], H, G, 64, 64, dtype, strided=True)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_continued_padded_and_empty(dtype):
    _check([40, 0, 1, 129, 3, 260], 2, 1, 32, 64, dtype, ctx=[0, 5, 700, 128, 127, 1], slots=[3, 2, 6, -1, 0, 5], tail=30)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_segments_of_a_long_prompt(dtype):
    # few heads, many tokens: the plan cuts the sequences
    assert kda.kda_ssm_scan_workspace_size(1, 2100, 2, 1, 32, 32, 0) > 0
    _check([2100], 2, 1, 32, 32, dtype)
    _check([1500, 3, 600], 2, 2, 16, 64, dtype, ctx=[77, 0, 300], slots=[1, 0, 4])


@pytest.mark.parametrize("lens,over", [([70, 200], dict(ctx=[5, 130], page=128)), ([33], {}), ([49, 0, 1, 700], dict(ctx=[15, 0, 16, 17])),
                                       ([130, 130], dict(packed=False, ctx=[127, 0], page=128)), ([1, 2, 400, 3], dict(slots=[0, -1, 2, 3]))])
@pytest.mark.parametrize("N,P", [(16, 16), (64, 32), (128, 128)])
def test_short_segments_in_fp32(lens, over, N, P):
    # the CUDA-core kernel's segments may be as short as 16 tokens
    _check(lens, 2, 1, N, P, F32, **over)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("page", [128, 256])
def test_snapshots(page, dtype):
    _check([300, 128, 20, 513], 2, 1, 16, 32, dtype, ctx=[0, 128, 110, 700], page=page)
    _check([1300], 2, 1, 16, 32, dtype, ctx=[60], page=page)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("over", [dict(softplus=False), dict(D=False), dict(bias=False), dict(state=False), dict(packed=False),
                                  dict(packed=False, ctx=[3, 0, 9]), dict(slow=0.01), dict(slow=3.0)])
def test_options(over, dtype):
    _check([140, 140, 140], 3, 1, 32, 32, dtype, **over)


@pytest.mark.parametrize("N,P", [(16, 16), (64, 128), (128, 64), (32, 32), (128, 16)])
@pytest.mark.parametrize("lens,over", [([16, 1, 9, 12, 16], {}), ([16, 0, 15, 1], dict(ctx=[0, 3, 500, 9], slots=[1, 0, -1, 4], tail=7)),
                                       ([1] * 70, dict(ctx=[5] * 70)), ([4] * 40, dict(packed=False, ctx=[0, 1] * 20)),
                                       ([2, 1, 3] * 50, {}), ([9, 16, 3], dict(ctx=[119, 127, 253], page=128)),
                                       ([2] * 64, dict(ctx=[126, 127] * 32, page=128))])
def test_few_tokens(lens, over, N, P):
    # sequences of up to 16 tokens are computed in fp32, whichever kernel takes the call
    _check(lens, 3, 1 if P > 16 else 3, N, P, BF, once=True, strided=over.get("packed", True), **over)


@pytest.mark.parametrize("N,P", [(16, 16), (64, 128), (128, 64)])
@pytest.mark.parametrize("lens", [[5, 300, 16, 17, 0, 1], [1029], [1, 640, 1, 1, 1, 1, 1, 1]])
def test_few_tokens_beside_many(lens, N, P):
    _check(lens, 2, 1, N, P, BF, ctx=[0, 130, 4, 0, 1, 127, 0, 0][:len(lens)])


def test_many_heads_of_a_batch():
    _check([150, 90], 80, 2, 128, 64, BF, strided=True)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("R,H,G,N,P", [(1, 32, 2, 128, 64), (7, 3, 1, 16, 16), (5, 4, 2, 64, 128), (33, 2, 1, 128, 128)])
def test_step(R, H, G, N, P, dtype):
    v = _inputs(R, H, G, N, P, dtype, R + N, R + 2)
    g = np.random.default_rng(R)
    sl = g.permutation(R + 2)[:R].astype(np.int32)
    if R > 2:
        sl[2] = -1
    d = {k: t.cuda() for k, t in v.items()}
    y = torch.full((R, H, P), 7.0, dtype=dtype, device="cuda")
    kda.ssm_step(d["x"], d["dt"], d["A"], d["B"], d["C"], d["state"], d["D"], d["dt_bias"], slots=torch.from_numpy(sl).cuda(), y=y)
    torch.cuda.synchronize()
    n = {k: _n(t) for k, t in v.items()}
    kw = dict(slots=sl, ctx=np.ones(R), R=R)
    ry, rs, _ = serving.ssm_scan(**n, **kw)
    ytol, stol, _ = _tolerances(n, kw, 1, N, F32, ry, rs, None)
    ytol = ytol + torch.finfo(dtype).eps / 2 * np.abs(ry)
    yn, seen = y.double().cpu().numpy(), sl >= 0
    assert (yn[~seen] == 7.0).all()
    assert (np.abs(yn - ry)[seen] <= ytol[seen]).all()
    assert (np.abs(d["state"].double().cpu().numpy() - rs) <= stol).all()


def test_steps_continue_a_prompt():
    v = _inputs(50, 4, 1, 64, 64, F32, 5, 1)
    d = {k: t.cuda() for k, t in v.items()}
    pool = torch.zeros(1, 4, 64, 64, device="cuda")
    at = lambda a, b: [d[k][a:b] for k in ("x", "dt")] + [d["A"]] + [d[k][a:b] for k in ("B", "C")]
    y = [kda.ssm_scan(*at(0, 40), d["D"], d["dt_bias"], state=pool)]
    y += [kda.ssm_step(*at(t, t + 1), pool, d["D"], d["dt_bias"]) for t in range(40, 50)]
    n = {k: _n(t) for k, t in v.items()}
    n["state"] = np.zeros((1, 4, 64, 64))
    ry, rs, _ = serving.ssm_scan(**n, R=1)
    ytol, stol, _ = _tolerances(n, dict(R=1), 50, 64, F32, ry, rs, None)
    assert (np.abs(torch.cat(y).double().cpu().numpy() - ry) <= ytol).all()
    assert (np.abs(pool.double().cpu().numpy() - rs) <= stol).all()


def test_values_outside_are_not_followed():
    v = {k: t.cuda() for k, t in _inputs(300, 2, 1, 16, 16, F32, 1, 2).items()}
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")
    run = lambda **kw: kda.ssm_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], **kw)
    y = torch.full((300, 2, 16), 7.0, device="cuda")
    before = v["state"].clone()
    run(state=v["state"], slots=i32([1, 2]), cu=i32([0, 100, 300]), y=y)
    assert kda.kda_get_device_status() == 10
    assert (y[100:] == 7).all() and (y[:100] != 7).any() and torch.equal(v["state"][0], before[0])
    y.fill_(7.0)
    run(cu=i32([0, 100, 301]), y=y)
    assert kda.kda_get_device_status() == 10
    assert (y[100:] == 7).all()
    pages = torch.zeros(1, 2, 16, 16, device="cuda")
    run(block_table=i32([[1, 0, -1]]), pages=pages, page_size=128)
    assert kda.kda_get_device_status() == 10
    assert pages.abs().sum() > 0
