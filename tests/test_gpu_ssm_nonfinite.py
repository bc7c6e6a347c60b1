"""A value that is not finite, in the middle of a sequence, against the same call
without it: which outputs stay as they were, bit for bit."""
import pytest
import torch

from gated_delta_rule_117_b200 import kda

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,T,H", [(BF, 300, 2), (BF, 2000, 1), (F32, 300, 2)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [5, 37, 127, 128, 200, 255, 290])
@pytest.mark.parametrize("which", ["x", "dt", "B", "C"])
def test_earlier_tokens(which, at, bad, dtype, T, H):
    N, P = 32, 64
    g = torch.Generator().manual_seed(T)
    rn = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()
    v = dict(x=rn(T, H, P), dt=rn(T, H), B=rn(T, 1, N), C=rn(T, 1, N))
    A, bias, ctx = -torch.rand(H, generator=g).cuda() - 0.5, torch.full((H,), -3.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    pages = torch.zeros(2, T // 128, H, N, P, device="cuda")
    table = torch.arange(T // 128, dtype=torch.int32, device="cuda")[None]

    def run(k):
        return kda.ssm_scan(v["x"], v["dt"], A, v["B"], v["C"], dt_bias=bias, ctx=ctx, block_table=table, pages=pages[k], page_size=128)

    clean = run(0)
    v[which][at] = bad
    y = run(1)
    first = at - at % 32 if which == "x" and dtype is BF else at  # (on the tensor cores 0 times x reaches its block of 32)
    assert torch.equal(y[:first], clean[:first])
    if which == "C":  # its own token's output only
        assert torch.equal(y[at + 1:], clean[at + 1:]) and torch.equal(pages[0], pages[1])
    k = at // 128  # states at positions up to it
    assert torch.equal(pages[1, :k], pages[0, :k]) and kda.kda_get_device_status() == 0
    assert not torch.isfinite(y[at].float()).all()
