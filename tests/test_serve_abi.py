"""Host-side checks of the packed-request operators (no GPU): every bad argument
is refused with its documented status code before any device call, and the
Python helpers name what is wrong with a tensor."""
import pytest
import torch

from gated_delta_rule_117_b200 import build as kbuild
from gated_delta_rule_117_b200 import kda

INVALID, SHAPE, DTYPE, ALIGN, ALIAS, WORKSPACE = 1, 2, 3, 4, 5, 6
BASE = 1 << 40  # never dereferenced
MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    kbuild.build()
    return kda.load_library()


def _passes(status):
    """Right arguments: on a machine without a GPU only the device check fails."""
    return status in (0, 7, 9) if not torch.cuda.is_available() else status in (0, 7)


def _map(**over):
    a = dict(length=BASE, ctx=BASE + MB, free_pages=BASE + 2 * MB, n_free=8, block_table=BASE + 3 * MB, table_stride=4,
             page_size=16, cu=BASE + 4 * MB, token_slots=BASE + 5 * MB, pages_used=BASE + 6 * MB, R=3, rows=40, stream=None)
    a.update(over)
    return kda.kda_block_map(**a)


@pytest.mark.parametrize("over,code", [
    (dict(R=-1), INVALID), (dict(rows=-1), INVALID), (dict(n_free=-1), INVALID), (dict(table_stride=-1), INVALID),
    (dict(page_size=0), INVALID), (dict(length=None), INVALID), (dict(cu=None), INVALID), (dict(token_slots=None), INVALID),
    (dict(pages_used=None), INVALID), (dict(block_table=None), INVALID), (dict(free_pages=None), INVALID),
    (dict(R=16385), SHAPE), (dict(length=BASE + 2), ALIGN), (dict(cu=BASE + 4 * MB + 2), ALIGN),
    (dict(token_slots=BASE + 5 * MB + 4), ALIGN), (dict(cu=BASE), ALIAS), (dict(token_slots=BASE + 2 * MB), ALIAS),
    (dict(pages_used=BASE + 4 * MB + 12), ALIAS), (dict(block_table=BASE + MB), ALIAS),
])
def test_block_map_rejects(over, code):
    assert _map(**over) == code


def _conv(**over):
    a = dict(x=BASE, x_stride=64, w=BASE + MB, bias=BASE + 2 * MB, state=BASE + 3 * MB, n_slots=4, slots=BASE + 4 * MB,
             ctx=BASE + 5 * MB, cu=BASE + 6 * MB, y=BASE + 7 * MB, y_stride=64, R=3, rows=30, C=64, K=4, head_dim=0, dtype=1,
             flags=1, eps=1e-6, stream=None)
    a.update(over)
    return kda.kda_short_conv(**a)


@pytest.mark.parametrize("over,code", [
    (dict(R=-1), INVALID), (dict(rows=-1), INVALID), (dict(C=-1), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(y=None), INVALID), (dict(state=None), INVALID), (dict(n_slots=0), INVALID), (dict(flags=8), INVALID),
    (dict(flags=3, head_dim=32, eps=float("nan")), INVALID), (dict(flags=3, head_dim=32, eps=-1.0), INVALID),
    (dict(flags=4, head_dim=32), INVALID),                       # head-major of packed rows
    (dict(K=1), SHAPE), (dict(K=5), SHAPE), (dict(x_stride=63), SHAPE), (dict(y_stride=63), SHAPE),
    (dict(flags=2, head_dim=24), SHAPE), (dict(flags=2, head_dim=128), SHAPE), (dict(cu=None, rows=31), SHAPE),
    (dict(slots=None, n_slots=2), SHAPE), (dict(C=(1 << 24) + 64, x_stride=1 << 25, y_stride=1 << 25), SHAPE),
    (dict(dtype=2), DTYPE), (dict(x=BASE + 1), ALIGN), (dict(slots=BASE + 4 * MB + 2), ALIGN), (dict(cu=BASE + 6 * MB + 1), ALIGN),
    (dict(y=BASE), ALIAS), (dict(y=BASE + 3 * MB), ALIAS), (dict(state=BASE + MB), ALIAS), (dict(y=BASE + 29 * 64 * 2 + 126), ALIAS),
])
def test_short_conv_rejects(over, code):
    assert _conv(**over) == code


@pytest.mark.parametrize("over", [{}, dict(bias=None), dict(state=None, n_slots=0), dict(ctx=None, slots=None), dict(cu=None),
                                  dict(x=BASE + 2, x_stride=65), dict(cu=None, flags=7, head_dim=16, y_stride=0)])
def test_short_conv_accepts(over):
    assert _passes(_conv(**over))


def _conv_step(**over):
    a = dict(x=BASE, x_stride=64, w=BASE + MB, bias=BASE + 2 * MB, state=BASE + 3 * MB, n_slots=4, slots=BASE + 4 * MB,
             y=BASE + 7 * MB, y_stride=64, R=3, C=64, K=4, head_dim=0, dtype=1, flags=1, eps=1e-6, stream=None)
    a.update(over)
    return kda.kda_short_conv_step(**a)


@pytest.mark.parametrize("over,code", [
    (dict(R=-1), INVALID), (dict(state=None, n_slots=0), INVALID), (dict(K=7), SHAPE), (dict(y_stride=10), SHAPE),
    (dict(slots=None, n_slots=2), SHAPE), (dict(dtype=9), DTYPE), (dict(w=BASE + MB + 1), ALIGN), (dict(y=BASE), ALIAS),
    (dict(state=BASE + 7 * MB), ALIAS),
])
def test_short_conv_step_rejects(over, code):
    assert _conv_step(**over) == code


def _scan(**over):
    a = dict(x=BASE, x_stride=256, dt=BASE + MB, dt_stride=4, A=BASE + 2 * MB, B=BASE + 3 * MB, b_stride=64, C=BASE + 4 * MB,
             c_stride=64, D=BASE + 5 * MB, dt_bias=BASE + 6 * MB, softplus=1, state=BASE + 7 * MB, n_slots=4,
             slots=BASE + 8 * MB, ctx=BASE + 9 * MB, cu=BASE + 10 * MB, block_table=BASE + 11 * MB, table_stride=2,
             pages=BASE + 12 * MB, n_pages=4, page_size=128, y=BASE + 14 * MB, y_stride=256, R=3, rows=30, H=4, G=2, N=32, P=64,
             dtype=1, workspace=None, workspace_bytes=0, stream=None)
    a.update(over)
    return kda.kda_ssm_scan(**a)


@pytest.mark.parametrize("over,code", [
    (dict(R=-1), INVALID), (dict(H=-4), INVALID), (dict(x=None), INVALID), (dict(dt=None), INVALID), (dict(A=None), INVALID),
    (dict(B=None), INVALID), (dict(C=None), INVALID), (dict(y=None), INVALID), (dict(state=None), INVALID),
    (dict(page_size=64), INVALID), (dict(page_size=-128), INVALID), (dict(block_table=None), INVALID),
    (dict(pages=None), INVALID), (dict(table_stride=-1), INVALID),
    (dict(N=24), SHAPE), (dict(P=256), SHAPE), (dict(G=3), SHAPE), (dict(G=0), SHAPE), (dict(x_stride=255), SHAPE),
    (dict(dt_stride=3), SHAPE), (dict(b_stride=63), SHAPE), (dict(c_stride=63), SHAPE), (dict(y_stride=255), SHAPE),
    (dict(cu=None, rows=31), SHAPE), (dict(slots=None, n_slots=2), SHAPE), (dict(R=1 << 28, H=4, n_slots=1), SHAPE),
    (dict(dtype=5), DTYPE), (dict(state=BASE + 7 * MB + 8), ALIGN), (dict(pages=BASE + 12 * MB + 8), ALIGN),
    (dict(A=BASE + 2 * MB + 2), ALIGN), (dict(x=BASE + 1), ALIGN), (dict(block_table=BASE + 11 * MB + 2), ALIGN),
    (dict(y=BASE), ALIAS), (dict(state=BASE + 3 * MB), ALIAS), (dict(pages=BASE + 7 * MB), ALIAS), (dict(y=BASE + 12 * MB), ALIAS),
])
def test_ssm_scan_rejects(over, code):
    assert _scan(**over) == code


def test_ssm_scan_workspace():
    need = kda.kda_ssm_scan_workspace_size(1, 100000, 4, 2, 32, 64, 1)
    assert need > 0 and need % 16 == 0
    long = dict(R=1, rows=100000, cu=None, page_size=0, slots=None, ctx=None, y=BASE + 1024 * MB, x=BASE + 512 * MB,
                dt=BASE + 400 * MB, B=BASE + 300 * MB, C=BASE + 200 * MB)
    assert _scan(**long) == WORKSPACE
    assert _scan(**long, workspace=BASE + 2048 * MB, workspace_bytes=need - 1) == WORKSPACE
    assert _scan(**long, workspace=BASE + 2048 * MB + 8, workspace_bytes=need) == ALIGN
    assert _scan(**long, workspace=BASE + 512 * MB, workspace_bytes=need) == ALIAS
    assert _passes(_scan(**long, workspace=BASE + 2048 * MB, workspace_bytes=need))
    bad = (1 << 64) - 1
    assert kda.kda_ssm_scan_workspace_size(1, 100, 4, 2, 33, 64, 1) == bad
    assert kda.kda_ssm_scan_workspace_size(-1, 100, 4, 2, 32, 64, 1) == bad
    assert kda.kda_ssm_scan_workspace_size(1, 100, 4, 3, 32, 64, 1) == bad
    assert kda.kda_ssm_scan_workspace_size(0, 0, 4, 2, 32, 64, 1) == 0


@pytest.mark.parametrize("R,rows", [(1, 5000), (3, 40000), (64, 64 * 300), (200, 1 << 20), (1, 1 << 20), (7, 130)])
def test_workspace_holds_every_segment(R, rows):
    # states and decays of `items` segments; items never fall short of the sequences' segments (for any cut of
    # the rows into sequences, and any ctx), as the numbering of the segments leaves room for them
    import random
    H, N, P = 2, 32, 64
    rng = random.Random(R)
    for seg in (128, 512, 896, 4096):
        items = rows // seg + 2 * R
        cuts = sorted(rng.randint(0, rows) for _ in range(R - 1))
        cu = [0] + cuts + [rows]
        base = [cu[r] // seg + 2 * r for r in range(R + 1)]
        for r in range(R):
            off, n = rng.choice([0, 1, 127]), cu[r + 1] - cu[r]
            count = -(-(off + n) // seg) if n else 0
            assert base[r] + count <= base[r + 1] <= items
    assert kda.kda_ssm_scan_workspace_size(R, rows, H, 1, N, P, 1) % 16 == 0


def _step(**over):
    a = dict(x=BASE, x_stride=256, dt=BASE + MB, dt_stride=4, A=BASE + 2 * MB, B=BASE + 3 * MB, b_stride=64, C=BASE + 4 * MB,
             c_stride=64, D=BASE + 5 * MB, dt_bias=BASE + 6 * MB, softplus=1, state=BASE + 7 * MB, n_slots=4,
             slots=BASE + 8 * MB, y=BASE + 14 * MB, y_stride=256, R=3, H=4, G=2, N=32, P=64, dtype=1, stream=None)
    a.update(over)
    return kda.kda_ssm_step(**a)


@pytest.mark.parametrize("over,code", [
    (dict(R=-1), INVALID), (dict(state=None, n_slots=0), INVALID), (dict(x=None), INVALID), (dict(N=8), SHAPE), (dict(G=3), SHAPE),
    (dict(y_stride=4), SHAPE), (dict(slots=None, n_slots=2), SHAPE), (dict(dtype=4), DTYPE), (dict(state=BASE + 7 * MB + 4), ALIGN),
    (dict(y=BASE + 8), ALIAS), (dict(state=BASE + 14 * MB), ALIAS),
])
def test_ssm_step_rejects(over, code):
    assert _step(**over) == code


def test_sizes_that_would_not_fit_their_arithmetic():
    most = (1 << 31) - 4097
    assert _conv(rows=most + 1) == SHAPE and _map(rows=most + 1) == SHAPE and _scan(rows=most + 1) == SHAPE
    assert _conv(x_stride=1 << 48) == SHAPE and _scan(x_stride=1 << 48) == SHAPE and _scan(dt_stride=1 << 48) == SHAPE
    assert _conv_step(y_stride=1 << 48) == SHAPE and _step(c_stride=1 << 48) == SHAPE


def test_heads_that_would_not_fit_their_arithmetic():
    most, far = 1 << 24, 1 << 36  # a place in a row is h * 128 + c in 32 bits
    wide = dict(G=1, N=16, P=128, R=1, x_stride=far, y_stride=far, dt_stride=far, n_slots=1)
    assert _step(H=most + 1, **wide) == SHAPE and _scan(H=most + 1, rows=1, **wide) == SHAPE
    assert _step(H=1 << 24, **dict(wide, R=128, n_slots=128)) == SHAPE  # and the blocks of a launch
    bad = (1 << 64) - 1
    assert kda.kda_ssm_scan_workspace_size(1, 1, most + 1, 1, 16, 128, 1) == bad
    assert kda.kda_ssm_scan_workspace_size(1 << 30, (1 << 31) - 4097, 1 << 20, 1, 128, 128, 1) == bad
    assert kda.kda_ssm_scan_workspace_size(1, (1 << 31) - 4096, 1, 1, 128, 128, 1) == bad


def test_nothing_to_do():
    assert _conv(R=0, rows=0, x=None) == 0 and _conv(rows=0, y=None) == 0 and _conv_step(R=0) == 0
    assert _scan(R=0, rows=0, x=None) == 0 and _scan(H=0, y=None) == 0 and _step(R=0) == 0


def test_helpers_refuse_host_tensors_and_wrong_types():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 4, dtype=torch.bfloat16)
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.short_conv(x, w)
    with pytest.raises(TypeError, match="w must be bfloat16"):
        kda.short_conv(x, w.float())
    with pytest.raises(TypeError):
        kda.short_conv(x.half(), w.half())
    with pytest.raises(ValueError, match="CUDA"):
        kda.short_conv_step(x, w, torch.zeros(4, 3, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        kda.block_map(i32, None, i32, torch.zeros(4, 2, dtype=torch.int32), 16, 8)
    with pytest.raises(TypeError, match="lens must be int32"):
        kda.block_map(i32.long(), None, i32, torch.zeros(4, 2, dtype=torch.int32), 16, 8)
    a = torch.zeros(2)
    z = lambda *s: torch.zeros(*s)
    with pytest.raises(ValueError, match="CUDA"):
        kda.ssm_scan(z(5, 2, 16), z(5, 2), a, z(5, 1, 16), z(5, 1, 16))
    with pytest.raises(TypeError, match="dt must be float32"):
        kda.ssm_step(z(5, 2, 16), z(5, 2).bfloat16(), a, z(5, 1, 16), z(5, 1, 16), z(5, 2, 16, 16))
    with pytest.raises(ValueError, match="x must be"):
        kda.ssm_step(z(2, 16), z(5, 2), a, z(5, 1, 16), z(5, 1, 16), z(5, 2, 16, 16))
