"""Short causal convolution (kda_short_conv, kda_short_conv_step) against the
fp64 oracle, element by element.

Tolerance.  v = bias + sum of K products is K fused operations in fp32: off by
at most (K + 1) 2^-24 M, M = |bias| + sum |w u|.  Swish has a slope below 1.1
and its own evaluation is off by at most 2^-20 |v| (the fast exponential and
division of the bf16 form; 2^-22 in fp32).  The norm divides by
n = sqrt(sum v^2 + eps): with every v of the head off by at most e, y is off by
at most (e + |y| sqrt(d) e) / n, and its square root and division add 4 2^-24.
The result is rounded once: half a step of the type, relative to the value.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_117_b200 import kda
from oracle import serving

pytestmark = pytest.mark.gpu

EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32


def _close(y, ref, x, w, bias, old, seqs, dtype, d, norm):
    """seqs: (lo, hi, old inputs or zeros) of every sequence that was computed."""
    K, C = w.shape[1], w.shape[0]
    half = torch.finfo(dtype).eps / 2
    seen = np.zeros(len(ref), bool)
    for lo, hi, before in seqs:
        seen[lo:hi] = True
        u = np.abs(np.concatenate([before, x[lo:hi]]))
        M = np.abs(bias)[None] + sum(np.abs(w[:, i])[None] * u[i:i + hi - lo] for i in range(K))
        e = 1.1 * (K + 1) * 2.0 ** -24 * M + (2.0 ** -20 if dtype == BF else 2.0 ** -22) * M
        r = ref[lo:hi]
        if norm:
            # n from the un-normalised reference: |v| <= M
            eh = e.reshape(len(r), -1, d).max(2)
            v, _ = serving.short_conv(np.concatenate([before, x[lo:hi]]), w, bias)
            n = np.sqrt((v[K - 1:].reshape(len(r), -1, d) ** 2).sum(2) + EPS)
            rep = lambda t: np.repeat(t, d, 1)
            e = (rep(eh) * (1 + np.abs(r) * np.sqrt(d))) / rep(n) + 4 * 2.0 ** -24 * np.abs(r)
        tol = e + half * (np.abs(r) + e)
        assert (np.abs(y[lo:hi] - r) <= tol).all(), float((np.abs(y[lo:hi] - r) / tol).max())
    return seen


def _run(lens, C, K, dtype, *, ctx=True, slots=True, packed=True, norm=False, head_major=False, d=0, silu=True, bias=True,
         pad=0, seed=0, tail=0, front=0):
    g = torch.Generator().manual_seed(seed + 17 * C + K)
    R, rows = len(lens), sum(lens)
    wide = torch.randn(front + rows + tail, C + pad, generator=g).to(dtype)
    wide[:front] = float("nan")
    wide[front + rows:] = float("nan")  # rows of no sequence must not be read
    w = (torch.randn(C, K, generator=g) / K ** 0.5).to(dtype)
    b = (0.1 * torch.randn(C, generator=g)).to(dtype) if bias else None
    pool = torch.randn(R + 2, K - 1, C, generator=g).to(dtype)
    c = torch.randint(0, 3, (R,), generator=g, dtype=torch.int32) if ctx else None
    sl = torch.randperm(R + 2, generator=g)[:R].to(torch.int32) if slots else None
    if slots and R > 2:
        sl[R // 2] = -1  # a padded request
    cu = (front + torch.tensor([0] + list(np.cumsum(lens)))).to(torch.int32) if packed else None
    x = wide.cuda()[:, :C]
    if not packed:
        x = x.unflatten(0, (R, -1))
    dev = lambda t: None if t is None else t.cuda()
    poold = pool.cuda()
    y0 = None
    if not head_major:
        y0 = torch.full(wide.shape, 7.0, dtype=dtype, device="cuda")[:, :C]
        y0 = y0.unflatten(0, (R, -1)) if not packed else y0
    y = kda.short_conv(x, w.cuda(), dev(b), state=poold, slots=dev(sl), ctx=dev(c), cu=dev(cu), silu=silu, head_dim=d,
                       l2norm=norm, head_major=head_major, eps=EPS, y=y0)
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == 0
    f = lambda t: None if t is None else t.double().numpy()
    xn = f(wide[:, :C])
    ref, rpool = serving.short_conv(xn, f(w), f(b), f(pool), None if sl is None else sl.numpy(),
                                    None if c is None else c.numpy(), None if cu is None else cu.numpy(), R, silu, d,
                                    EPS if norm else None)
    assert torch.equal(poold.cpu().double(), torch.from_numpy(rpool))  # inputs are moved, not computed
    yn = y.double().cpu().numpy()
    if head_major:
        yn = yn.transpose(0, 2, 1, 3).reshape(rows, C)
    yn = yn.reshape(len(xn), C)
    seqs, lo = [], front
    for r, n in enumerate(lens):
        if (sl is None or sl[r] >= 0) and n:
            carried = c is not None and c[r] > 0
            seqs.append((lo, lo + n, f(pool[r if sl is None else sl[r]]) if carried else np.zeros((K - 1, C))))
        lo += n
    seen = _close(yn, ref, xn, f(w), np.zeros(C) if b is None else f(b), None, seqs, dtype, d, norm)
    if not head_major:
        assert (yn[~seen] == 7.0).all()  # rows of no sequence and of padded requests


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C,pad", [(1, 0), (7, 0), (40, 8), (515, 1), (2048, 16)])
def test_packed(C, pad, dtype, K):
    _run([1, 0, 2, 37, 3, 16, 15, 17, 100, 0], C, K, dtype, pad=pad)


@pytest.mark.parametrize("seed", range(12))
def test_sequences_across_tiles(seed):
    # many short sequences around the tiles' borders, continued from the pool
    g = np.random.default_rng(seed)
    _run(list(g.integers(0, 7 if seed % 2 else 40, 60)), 24, 2 + seed % 3, BF, seed=seed, tail=seed % 4 * 9, front=seed % 3 * 5)


@pytest.mark.parametrize("d,H", [(16, 1), (16, 5), (32, 3), (64, 2), (128, 3), (128, 16)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm,head_major", [(True, False), (True, True), (False, True)])
def test_heads(norm, head_major, dtype, d, H):
    _run([53] * 3, d * H, 4, dtype, norm=norm, head_major=head_major, d=d, packed=False, pad=8)


@pytest.mark.parametrize("over", [dict(silu=False), dict(bias=False), dict(ctx=False), dict(slots=False), dict(tail=40)])
def test_options(over):
    _run([30, 1, 80], 96, 4, BF, **over)


def test_norm_of_misaligned_rows():
    # a row stride of an odd number of elements: element-wise loads, the same lanes for a head
    _run([20, 33], 128, 4, BF, norm=True, d=64, pad=3)


def test_without_pool():
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn(2, 19, 32, generator=g), torch.randn(32, 3, generator=g)
    y = kda.short_conv(x.cuda(), w.cuda())
    ref, _ = serving.short_conv(x.reshape(38, 32).double().numpy(), w.double().numpy(), None, R=2)
    xs = x.reshape(38, 32).double().numpy()
    _close(y.double().cpu().numpy().reshape(38, 32), ref, xs, w.double().numpy(), np.zeros(32), None,
           [(0, 19, np.zeros((2, 32))), (19, 38, np.zeros((2, 32)))], F32, 0, False)


@pytest.mark.parametrize("R,C,K,dtype,norm,d", [(1, 2048, 4, BF, True, 128), (256, 4352, 4, BF, False, 0), (5, 515, 3, F32, False, 0),
                                               (3, 1, 2, BF, False, 0), (9, 96, 4, F32, True, 32), (2, 80, 2, BF, True, 16)])
def test_step(R, C, K, dtype, norm, d):
    g = torch.Generator().manual_seed(R + C)
    x = torch.randn(R, C + 8, generator=g).to(dtype)
    w = (torch.randn(C, K, generator=g) / K ** 0.5).to(dtype)
    b = (0.1 * torch.randn(C, generator=g)).to(dtype)
    pool = torch.randn(R + 2, K - 1, C, generator=g).to(dtype)
    sl = torch.randperm(R + 2, generator=g)[:R].to(torch.int32)
    if R > 2:
        sl[1] = -1
    poold, y0 = pool.cuda(), torch.full((R, C), 7.0, dtype=dtype, device="cuda")
    y = kda.short_conv_step(x.cuda()[:, :C], w.cuda(), poold, b.cuda(), slots=sl.cuda(), head_dim=d, l2norm=norm, eps=EPS, y=y0)
    torch.cuda.synchronize()
    f = lambda t: t.double().numpy()
    ref, rpool = serving.short_conv(f(x[:, :C]), f(w), f(b), f(pool), sl.numpy(), np.ones(R), None, R, True, d, EPS if norm else None)
    assert torch.equal(poold.cpu().double(), torch.from_numpy(rpool))
    yn = y.double().cpu().numpy()
    seqs = [(r, r + 1, f(pool[sl[r]])) for r in range(R) if sl[r] >= 0]
    seen = _close(yn, ref, f(x[:, :C]), f(w), f(b), None, seqs, dtype, d, norm)
    assert (yn[~seen] == 7.0).all()


def test_steps_continue_a_prompt():
    # a prompt, then tokens one by one, equal the prompt that holds them all, bit for bit
    g = torch.Generator().manual_seed(8)
    x, w = torch.randn(1, 40, 256, generator=g).to(BF).cuda(), torch.randn(256, 4, generator=g).to(BF).cuda()
    kw = dict(head_dim=128, l2norm=True)
    whole = kda.short_conv(x, w, **kw)
    pool = torch.zeros(1, 3, 256, dtype=BF, device="cuda")
    parts = [kda.short_conv(x[:, :33], w, state=pool, **kw)[0]]
    parts += [kda.short_conv_step(x[:, t], w, pool, **kw) for t in range(33, 40)]
    assert torch.equal(torch.cat(parts), whole[0])


def test_values_outside_are_not_followed():
    x, w = torch.randn(6, 8, device="cuda"), torch.randn(8, 4, device="cuda")
    pool = torch.zeros(2, 3, 8, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    y = torch.full((6, 8), 7.0, device="cuda")
    kda.short_conv(x, w, state=pool, slots=i32([2, 1]), cu=i32([0, 3, 6]), y=y)  # slot 2 of a pool of 2
    assert kda.kda_get_device_status() == 10
    assert (y[:3] == 7).all() and (y[3:] != 7).all() and (pool[0] == 0).all()
    y.fill_(7.0)
    kda.short_conv(x, w, cu=i32([0, 3, 9]), y=y)  # rows behind the array
    assert kda.kda_get_device_status() == 10
    assert (y[:3] != 7).all() and (y[3:] == 7).all()
    kda.short_conv_step(x[:2], w, pool, slots=i32([5, -1]), y=y[:2])
    assert kda.kda_get_device_status() == 10 and kda.kda_get_device_status() == 0
