"""Failure detection of the tensor-core scan without a GPU fault: its bounded
waits run out (a barrier that nothing arrives on, a limit shorter than an ordinary
wait), the CTAs drain what is in flight and return, the status word tells, and the
next call is right."""
import pytest
import torch

from gated_delta_rule_117_b200 import kda

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
TIMEOUT = 8


def _inputs(rows, H, N, P):
    g = torch.Generator().manual_seed(rows + N)
    rn = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()
    return (rn(rows, H, P), rn(rows, H), -torch.rand(H, generator=g).cuda() - 0.5, rn(rows, 1, N), rn(rows, 1, N),
            torch.ones(H, device="cuda"), torch.full((H,), -3.0, device="cuda"))


def _with_limit(ns, stall, ins):
    kda.kda_debug_set_wait_limit(ns)
    kda.kda_debug_inject_stall(stall)
    try:
        kda.ssm_scan(*ins)
        return kda.kda_get_device_status()  # synchronises
    finally:
        kda.kda_debug_inject_stall(False)
        kda.kda_debug_set_wait_limit(0)


# one chunk, two (every load is in flight before the first wait of the producer), many, and segments
@pytest.mark.parametrize("rows", [100, 250, 700, 3000])
@pytest.mark.parametrize("N,P", [(16, 64), (128, 128)])
@pytest.mark.parametrize("ns,stall", [(5_000_000, True), (1, True), (1, False)])
def test_waits_that_run_out(ns, stall, N, P, rows):
    ins = _inputs(rows, 2, N, P)
    assert (kda.kda_ssm_scan_workspace_size(1, rows, 2, 1, N, P, kda.KDA_DTYPE_BF16) > 0) or rows < 3000
    ref = kda.ssm_scan(*ins)
    assert kda.kda_get_device_status() == 0
    for _ in range(3):
        code = _with_limit(ns, stall, ins)
        assert code == TIMEOUT if stall else code in (0, TIMEOUT)
        assert kda.kda_get_device_status() == 0  # reading the word cleared it
        assert torch.equal(kda.ssm_scan(*ins), ref)
    assert kda.kda_get_device_status() == 0
