"""The host plan of a scan: cheap beside the call that it is for, and the same
sizes whenever it is asked."""
import random
import time

import pytest

from gated_delta_rule_117_b200 import build as kbuild
from gated_delta_rule_117_b200 import kda


@pytest.fixture(scope="module", autouse=True)
def lib():
    kbuild.build()
    return kda.load_library()


def _us(*args):
    f, best = kda.load_library().kda_ssm_scan_workspace_size, 1e9
    for _ in range(60):
        t0 = time.perf_counter()
        for _ in range(200):
            f(*args)
        best = min(best, time.perf_counter() - t0)
    return best / 200 * 1e6


@pytest.mark.parametrize("args", [(1, 4096, 32, 1, 128, 64, 1), (1, 131072, 16, 1, 128, 128, 1), (1, 4000, 32, 1, 128, 128, 0)])
def test_size_query_costs_little(args):
    # against a query that plans nothing, i.e. the call itself: a search of every length took 7 to 9 times as long
    # (a busy machine gets three tries)
    assert any(_us(*args) < 4 * _us(0, 0, 4, 1, 128, 64, 1) for _ in range(3))


def test_sizes_hold_every_form():
    # enough for whole sequences and segments of each form; more sequences of the same rows need no less room each
    rng = random.Random(3)
    for _ in range(2000):
        R, H, G = rng.randint(1, 70), rng.choice([1, 2, 4, 32]), 1
        N, P = rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128])
        rows = rng.randint(0, 1 << rng.randint(1, 20))
        both = [kda.kda_ssm_scan_workspace_size(R, rows, H, G, N, P, t) for t in (0, 1)]
        assert both == [kda.kda_ssm_scan_workspace_size(R, rows, H, G, N, P, t) for t in (0, 1)]
        assert all(b % 16 == 0 for b in both) and both[1] >= both[0]  # bf16 may take either kernel
        # a segment is 16 tokens at least: states and decays of that many, and of two more a sequence
        assert both[0] <= (rows // 16 + 2 * R) * H * (N * P + 1) * 4 + 16
