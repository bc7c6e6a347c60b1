"""Block tables and token slots from request lengths (kda_block_map): every
output is whole numbers and equals the oracle's."""
import numpy as np
import pytest
import torch

from gated_delta_rule_117_b200 import kda
from oracle import serving

pytestmark = pytest.mark.gpu


def _case(R, most, page, seed, ctx=True, blocks=None, free=None):
    g = np.random.default_rng(seed)
    lens = g.integers(0, most + 1, R).astype(np.int32)
    lens[g.random(R) < 0.15] = 0
    c = g.integers(0, 4 * page + 3, R).astype(np.int32) * (g.random(R) < 0.7) if ctx else None
    cc = c if ctx else np.zeros(R, np.int64)
    need = int(sum(-(-(int(a) + int(b)) // page) - -(-int(a) // page) for a, b in zip(cc, lens)))
    width = int(max(-(-(int(a) + int(b)) // page) for a, b in zip(cc, lens))) if R else 0
    blocks = width + 1 if blocks is None else blocks
    ids = g.permutation(need + 4 * R * 5 + 8).astype(np.int32)
    pages = ids[:need + 3] if free is None else ids[:free]
    table = np.where(np.arange(blocks)[None] < -(-np.asarray(cc)[:, None] // page), g.integers(0, 1 << 20, (R, blocks)), -7)
    return lens, c, pages, table.astype(np.int32)


def _check(lens, ctx, free, table, page, rows):
    d = lambda v: None if v is None else torch.from_numpy(np.ascontiguousarray(v, dtype=np.int32)).cuda()
    tab = d(table)
    cu, slots, used = kda.block_map(d(lens), d(ctx), d(free), tab, page, rows)
    rc, rt, rs, ru = serving.block_map(lens, ctx, free, table, page, rows)
    assert cu.cpu().tolist() == rc.tolist()
    assert int(used) == ru
    assert torch.equal(tab.cpu(), torch.from_numpy(rt))
    assert torch.equal(slots.cpu(), torch.from_numpy(rs))
    assert kda.kda_get_device_status() == 0


@pytest.mark.parametrize("R,most,page,ctx", [(1, 1, 1, False), (1, 700, 16, True), (7, 50, 64, True), (255, 9, 16, True),
                                             (256, 1, 512, True), (257, 40, 3, False), (1000, 30, 64, True)])
def test_matches_oracle(R, most, page, ctx):
    lens, c, free, table = _case(R, most, page, R + page, ctx)
    _check(lens, c, free, table, page, int(lens.sum()))
    _check(lens, c, free, table, page, int(lens.sum()) + 1500)  # rows behind the last token
    _check(lens, c, free, table, page, int(lens.sum()) // 2)    # more tokens than rows


def test_too_few_blocks_or_columns():
    lens, c, free, table = _case(20, 60, 8, 5, free=11)
    _check(lens, c, free, table, 8, int(lens.sum()))
    lens, c, free, table = _case(20, 60, 8, 6, blocks=3)
    _check(lens, c, free, table, 8, int(lens.sum()))
    lens, c, free, table = _case(3, 60, 8, 7, blocks=0)
    _check(lens, c, free[:0], table, 8, int(lens.sum()))


def test_more_requests_than_a_block_has_threads_many_times():
    lens, c, free, table = _case(16384, 3, 2, 11)
    _check(lens, c, free, table, 2, int(lens.sum()))


def test_lengths_that_do_not_add_up_to_32_bits():
    # sums saturate, and nothing is written outside
    R = 4
    lens = np.array([5, 2**31 - 1, 2**31 - 1, 7], np.int32)
    d = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table = torch.full((R, 3), -9, dtype=torch.int32, device="cuda")
    cu, slots, used = kda.block_map(d(lens.tolist()), None, d(list(range(50))), table, 1, 40)
    assert cu.tolist() == [0, 5, 2**31 - 1, 2**31 - 1, 2**31 - 1] and int(used) == 2**31 - 1
    assert table.tolist() == [[0, 1, 2], [5, 6, 7], [-1] * 3, [-1] * 3]
    assert slots.tolist() == [0, 1, 2, -1, -1, 5, 6, 7] + [-1] * 32


def test_negative_lengths_count_as_none():
    lens, c, free, table = _case(9, 30, 8, 9)
    lens[3] = -5
    c[4] = -2
    _check(lens, c, free, table, 8, 400)


def test_no_requests():
    _check(np.zeros(0, np.int32), None, np.zeros(0, np.int32), np.zeros((0, 4), np.int32), 16, 5)


def test_replayed_graph_reads_new_lengths():
    R, page, rows = 12, 16, 600
    sets = [_case(R, 40, page, s, blocks=12) for s in (1, 2, 3)]
    n_free = min(len(s[2]) for s in sets)
    d = lambda v: torch.from_numpy(np.ascontiguousarray(v, dtype=np.int32)).cuda()
    lens, ctx, free, table = (d(v[:n_free] if i == 2 else v) for i, v in enumerate(sets[0]))
    out = kda.block_map(lens, ctx, free, table, page, rows)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.block_map(lens, ctx, free, table, page, rows, cu=out[0], token_slots=out[1], pages_used=out[2])
    for s in sets[1:]:
        for t, v in zip((lens, ctx, free, table), (s[0], s[1], s[2][:n_free], s[3])):
            t.copy_(d(v))
        g.replay()
        ref = serving.block_map(s[0], s[1], s[2][:n_free], s[3], page, rows)
        assert out[0].cpu().tolist() == ref[0].tolist() and int(out[2]) == ref[3]
        assert torch.equal(table.cpu(), torch.from_numpy(ref[1])) and torch.equal(out[1].cpu(), torch.from_numpy(ref[2]))
