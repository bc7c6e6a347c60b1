"""The packed-request operators as a serving loop uses them together: request
lengths to offsets and block tables, convolution, scan with snapshots, then
single tokens, all against the fp64 oracle; the convolution as the input edge of
a KDA layer; two calls at once, replayed graphs, another stream, offsets beyond
32 bits, and values that must not leak from one request into another.

Tolerances: the operators' own element-wise ones are checked in their tests;
here whole tensors are compared (relative L2), bf16 within 3e-3 for each
rounded stage of the chain (half a bf16 step is 2^-9 = 2e-3 in the mean square),
fp32 within 1e-5.
"""
import numpy as np
import pytest
import torch

import oracle
from gated_delta_rule_117_b200 import kda
from oracle import serving
from parity_util import rel_l2

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TOL = {BF: 3e-3, F32: 1e-5}


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def _n(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prompts_then_tokens(dtype):
    # three rounds of a server: two of prompts (the second continues some), one of single tokens
    H, G, N, P, K, page = 4, 2, 64, 64, 4, 128
    C = H * P + 2 * G * N
    g = torch.Generator().manual_seed(7)
    rn = lambda *s: torch.randn(*s, generator=g)
    w, b = (rn(C, K) / 2).to(dtype), (0.1 * rn(C)).to(dtype)
    A, D, dt_bias = -(1 + 3 * torch.rand(H, generator=g)), 1 + 0.1 * rn(H), -3 + 0.5 * rn(H)
    R, blocks, n_pages = 5, 8, 40
    slots = torch.randperm(R + 2, generator=g)[:R].to(torch.int32)
    conv_pool, ssm_pool = torch.zeros(R + 2, K - 1, C, dtype=dtype), torch.zeros(R + 2, H, N, P)
    dev = dict(w=w.cuda(), b=b.cuda(), A=A.cuda(), D=D.cuda(), dt_bias=dt_bias.cuda(), conv=conv_pool.cuda(), ssm=ssm_pool.cuda(),
               pages=torch.zeros(n_pages, H, N, P, device="cuda"), table=torch.full((R, blocks), -1, dtype=torch.int32, device="cuda"),
               free=torch.randperm(n_pages, generator=g).to(torch.int32).cuda(), slots=slots.cuda())
    ref = dict(conv=_n(conv_pool), ssm=_n(ssm_pool), pages=np.zeros((n_pages, H, N, P)), table=np.full((R, blocks), -1),
               free=dev["free"].cpu().numpy())
    ctx = np.zeros(R, np.int64)
    for lens in ([300, 1, 0, 129, 70], [50, 200, 131, 0, 58]):
        rows = sum(lens)
        x, dt = rn(rows, C).to(dtype), rn(rows, H).to(dtype)
        cu, _, used = kda.block_map(_i32(lens), _i32(ctx), dev["free"], dev["table"], page, rows)
        dev["free"] = dev["free"][int(used):].contiguous()
        y = kda.short_conv(x.cuda(), dev["w"], dev["b"], state=dev["conv"], slots=dev["slots"], ctx=_i32(ctx), cu=cu)
        split = lambda t, lo, n, d: t[:, lo:lo + n * d].unflatten(1, (n, d))
        parts = split(y, 0, H, P), split(y, H * P, G, N), split(y, H * P + G * N, G, N)
        o = kda.ssm_scan(parts[0], dt.cuda(), dev["A"], parts[1], parts[2], dev["D"], dev["dt_bias"], state=dev["ssm"],
                         slots=dev["slots"], ctx=_i32(ctx), cu=cu, block_table=dev["table"], pages=dev["pages"], page_size=page)
        torch.cuda.synchronize()
        rcu, ref["table"], _, rused = serving.block_map(lens, ctx, ref["free"], ref["table"], page, rows)
        ref["free"] = ref["free"][rused:]
        assert cu.cpu().tolist() == rcu.tolist() and torch.equal(dev["table"].cpu().long(), torch.from_numpy(ref["table"]).long())
        ry, ref["conv"] = serving.short_conv(_n(x), _n(w), _n(b), ref["conv"], slots.numpy(), ctx, rcu, R)
        assert rel_l2(y, ry) <= TOL[dtype] and torch.equal(dev["conv"].double().cpu(), torch.from_numpy(ref["conv"]))
        q = _n(y)  # each stage is held to the oracle on its own inputs
        ro, ref["ssm"], ref["pages"] = serving.ssm_scan(
            q[:, :H * P].reshape(rows, H, P), _n(dt), _n(A), q[:, H * P:H * P + G * N].reshape(rows, G, N),
            q[:, H * P + G * N:].reshape(rows, G, N), _n(D), _n(dt_bias), True, ref["ssm"], slots.numpy(), ctx, rcu, R,
            ref["table"], ref["pages"], page)
        assert rel_l2(o, ro) <= TOL[dtype]
        assert rel_l2(dev["ssm"], ref["ssm"]) <= TOL[F32] and rel_l2(dev["pages"], ref["pages"]) <= TOL[F32]
        ctx = ctx + np.asarray(lens)
    for _ in range(4):  # single tokens
        x, dt = rn(R, C).to(dtype), rn(R, H).to(dtype)
        y = kda.short_conv_step(x.cuda(), dev["w"], dev["conv"], dev["b"], slots=dev["slots"])
        o = kda.ssm_step(split(y, 0, H, P), dt.cuda(), dev["A"], split(y, H * P, G, N), split(y, H * P + G * N, G, N), dev["ssm"],
                         dev["D"], dev["dt_bias"], slots=dev["slots"])
        torch.cuda.synchronize()
        ones = np.ones(R)
        ry, ref["conv"] = serving.short_conv(_n(x), _n(w), _n(b), ref["conv"], slots.numpy(), ones, None, R)
        assert rel_l2(y, ry) <= TOL[dtype]
        q = _n(y)
        ro, ref["ssm"], _ = serving.ssm_scan(q[:, :H * P].reshape(R, H, P), _n(dt), _n(A), q[:, H * P:H * P + G * N].reshape(R, G, N),
                                             q[:, H * P + G * N:].reshape(R, G, N), _n(D), _n(dt_bias), True, ref["ssm"],
                                             slots.numpy(), ones, None, R)
        assert rel_l2(o, ro) <= TOL[dtype] and rel_l2(dev["ssm"], ref["ssm"]) <= TOL[F32]
    # a snapshot resumes its sequence: request 0's state after 256 tokens, then its tokens behind it
    assert kda.kda_get_device_status() == 0


def test_resume_from_a_snapshot():
    H, N, P, page, T = 2, 128, 64, 128, 400
    g = torch.Generator().manual_seed(3)
    x, dt, B, C = (torch.randn(T, *s, generator=g).to(BF).cuda() for s in ((H, P), (H,), (1, N), (1, N)))
    A, bias = torch.tensor([-1.0, -4.0]).cuda(), torch.tensor([-3.0, -4.0]).cuda()
    pages, table = torch.zeros(4, H, N, P, device="cuda"), _i32([[2, 0, 3]])
    y = kda.ssm_scan(x, dt, A, B, C, dt_bias=bias, block_table=table, pages=pages, page_size=page)
    pool = pages[0:1].clone()  # after 256 tokens
    rest = kda.ssm_scan(x[256:], dt[256:], A, B[256:], C[256:], dt_bias=bias, state=pool, ctx=_i32([256]))
    # the state is the same fp32 values and the chunks are the same: bit for bit
    assert torch.equal(rest, y[256:])


@pytest.mark.parametrize("T", [90, 700])
def test_input_edge_of_a_kda_layer(T):
    # Eq. 2: q, k = L2Norm(Swish(ShortConv)), v = Swish(ShortConv), then the recurrence, prompt and one token
    B, H, d, K = 2, 3, 128, 4
    g = torch.Generator().manual_seed(T)
    rn = lambda *s: torch.randn(*s, generator=g)
    proj = rn(B, T + 1, 3 * H * d).to(BF).cuda()  # one projection for q, k and v
    ws = [(rn(H * d, K) / 2).to(BF) for _ in range(3)]
    gl, beta = -5 * torch.sigmoid(rn(B, H, T + 1, d)).to(BF), torch.sigmoid(rn(B, H, T + 1)).to(BF)
    pools = [torch.zeros(B, K - 1, H * d, dtype=BF, device="cuda") for _ in range(3)]
    S = torch.zeros(B, H, d, d, device="cuda")
    kw = [dict(head_dim=d, l2norm=n < 2) for n in range(3)]
    cut = lambda n: proj[..., n * H * d:(n + 1) * H * d]
    q, k, v = (kda.short_conv(cut(n)[:, :T].contiguous(), ws[n].cuda(), state=pools[n], head_major=True, **kw[n]) for n in range(3))
    at = lambda t, lo, hi: t[:, :, lo:hi].contiguous().cuda()
    o, _ = kda.chunk_fwd(q, k, v, at(gl, 0, T), at(beta, 0, T), h_T=S)
    q1, k1, v1 = (kda.short_conv_step(cut(n)[:, T], ws[n].cuda(), pools[n], **kw[n]).view(B, H, d) for n in range(3))
    one = lambda t: at(t, T, T + 1)[:, :, 0].contiguous()
    o1 = kda.recurrent_step(q1, k1, v1, one(gl), one(beta), S)
    torch.cuda.synchronize()
    ref = []
    for n in range(3):
        x = _n(cut(n)).reshape(B * (T + 1), H * d)
        y, _ = serving.short_conv(x, _n(ws[n]), None, R=B, head_dim=d, eps=1e-6 if n < 2 else None)
        ref.append(y.reshape(B, T + 1, H, d).transpose(0, 2, 1, 3))
    for got, one_got, r in zip((q, k, v), (q1, k1, v1), ref):
        assert rel_l2(got, r[:, :, :T]) <= TOL[BF] and rel_l2(one_got, r[:, :, T]) <= TOL[BF]
    cat = lambda a, b: np.concatenate([_n(a), _n(b)[:, :, None]], 2)
    ro, rS = oracle.recurrent(cat(q, q1), cat(k, k1), cat(v, v1), _n(gl), _n(beta))
    assert rel_l2(o, ro[:, :, :T]) <= TOL[BF] and rel_l2(o1, ro[:, :, T]) <= TOL[BF] and rel_l2(S, rS) <= TOL[BF]


def _scan_inputs(rows, H, N, P, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()
    return (rn(rows, H, P), rn(rows, H), -torch.rand(H, generator=g).cuda() - 0.5, rn(rows, 1, N), rn(rows, 1, N),
            torch.ones(H, device="cuda"), torch.full((H,), -3.0, device="cuda"))


@pytest.mark.parametrize("dtype,rows,H", [(BF, 6000, 2), (F32, 900, 2), (BF, 300, 64)])
def test_two_streams_at_once(dtype, rows, H):
    # segmented and whole calls that overlap, each with a workspace of its own, equal the calls alone
    ins = [_scan_inputs(rows, H, 64, 64, dtype, s) for s in range(4)]
    alone = [kda.ssm_scan(*i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    outs = [torch.zeros_like(a) for a in alone]
    for _ in range(5):
        for i, st, y in zip(ins, streams, outs):
            with torch.cuda.stream(st):
                kda.ssm_scan(*i, y=y)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, outs))
    # a stream that is handed over by name
    y = torch.zeros_like(alone[0])
    kda.ssm_scan(*ins[0], y=y, stream=streams[1])
    streams[1].synchronize()
    assert torch.equal(y, alone[0]) and kda.kda_get_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_replayed_graph_reads_new_lengths(dtype):
    # one graph of offsets, convolution, scan and a token step, replayed on other lengths, contexts and inputs
    H, G, N, P, K, rows, R = 2, 1, 64, 64, 4, 900, 4
    C = H * P + 2 * G * N
    g = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()
    w, A, bias = rn(C, K), -torch.rand(H, generator=g).cuda(), torch.full((H,), -3.0, device="cuda")
    x, dt, lens, ctx, slots = rn(rows, C), rn(rows, H), _i32([900, 0, 0, 0]), _i32([0] * R), _i32([3, 0, 2, 1])
    conv, ssm, table = torch.zeros(R, K - 1, C, dtype=dtype, device="cuda"), torch.zeros(R, H, N, P, device="cuda"), _i32([[-1] * 9] * R)
    free = _i32(range(40))

    def round_(out=None):
        cu, _, _ = kda.block_map(lens, ctx, free, table, 128, rows)
        y = kda.short_conv(x, w, state=conv, slots=slots, ctx=ctx, cu=cu)
        o = kda.ssm_scan(y[:, :H * P].unflatten(1, (H, P)), dt, A, y[:, H * P:H * P + N].unflatten(1, (1, N)),
                         y[:, H * P + N:].unflatten(1, (1, N)), dt_bias=bias, state=ssm, slots=slots, ctx=ctx, cu=cu)
        t = kda.ssm_step(o[:R], dt[:R], A, y[:R, H * P:H * P + N].unflatten(1, (1, N)), y[:R, H * P + N:].unflatten(1, (1, N)), ssm,
                         dt_bias=bias, slots=slots)
        return o, t

    round_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, t = round_()
    for lengths, c in (([900, 0, 0, 0], [0, 0, 0, 0]), ([10, 500, 1, 389], [5, 0, 128, 1000]), ([225] * 4, [0, 7, 0, 3])):
        seed = torch.randn(R, K - 1, C, generator=g).to(dtype).cuda()
        x.copy_(rn(rows, C)); dt.copy_(rn(rows, H)); lens.copy_(_i32(lengths)); ctx.copy_(_i32(c))
        conv.copy_(seed); ssm.fill_(0.25)
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in (o, t, conv, ssm)]
        conv.copy_(seed); ssm.fill_(0.25)
        eager = round_()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (*eager, conv, ssm)))
    assert kda.kda_get_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nothing_leaks_between_requests(dtype):
    # neighbours of NaN and infinities, padded requests of NaN, unread pool entries of NaN
    H, N, P, K = 2, 64, 64, 4
    lens = [5, 130, 77, 1, 200]
    rows, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)])
    x, dt, A, B, C, D, bias = _scan_inputs(rows, H, N, P, dtype, 9)
    clean = [t.clone() for t in (x, dt, B, C)]
    for r, bad in ((1, float("nan")), (3, float("inf"))):
        for t in (x, dt, B, C):
            t[cu[r]:cu[r + 1]] = bad
    pool = torch.full((7, H, N, P), float("nan"), device="cuda")
    pool[4] = 0.5
    slots, ctx = _i32([0, 1, -1, 3, 4]), _i32([0, 0, 9, 0, 40])  # only the last reads its entry
    x[cu[2]:cu[3]] = float("nan")
    y = torch.full_like(x, 7.0)
    kda.ssm_scan(x, dt, A, B, C, D, bias, state=pool, slots=slots, ctx=ctx, cu=_i32(cu), y=y)
    ref = torch.full_like(x, 7.0)
    pool2 = torch.zeros(7, H, N, P, device="cuda")
    pool2[4] = 0.5
    kda.ssm_scan(clean[0], clean[1], A, clean[2], clean[3], D, bias, state=pool2, slots=slots, ctx=ctx, cu=_i32(cu), y=ref)
    torch.cuda.synchronize()
    for r in (0, 2, 4):
        assert torch.equal(y[cu[r]:cu[r + 1]], ref[cu[r]:cu[r + 1]])
    for s in (0, 4):
        assert torch.equal(pool[s], pool2[s])
    assert torch.isnan(pool[[2, 5, 6]]).all()
    # the same for the convolution
    w = torch.randn(H * P, K, device="cuda").to(dtype)
    cpool = torch.full((7, K - 1, H * P), float("nan"), dtype=dtype, device="cuda")
    cpool[4] = 0.5
    c2 = cpool.clone()
    ya, yb = (torch.full((rows, H * P), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    kda.short_conv(x.flatten(1), w, state=cpool, slots=slots, ctx=ctx, cu=_i32(cu), y=ya)
    kda.short_conv(clean[0].flatten(1), w, state=c2, slots=slots, ctx=ctx, cu=_i32(cu), y=yb)
    torch.cuda.synchronize()
    for r in (0, 2, 4):
        assert torch.equal(ya[cu[r]:cu[r + 1]], yb[cu[r]:cu[r + 1]])
    assert torch.equal(cpool[0], c2[0]) and torch.equal(cpool[4], c2[4]) and torch.isnan(cpool[[2, 5, 6]].float()).all()


def test_offsets_beyond_32_bits():
    # more than 2^31 elements in x and y: the last sequence equals the same sequence alone
    C, rows = 4096, 540000
    x = torch.zeros(rows, C, dtype=BF, device="cuda")
    last = torch.randn(300, C, device="cuda").to(BF)
    x[-300:] = last
    w = torch.randn(C, 4, device="cuda").to(BF)
    cu = _i32([0, 7, rows - 300, rows])
    y = kda.short_conv(x, w, cu=cu)
    assert torch.equal(y[-300:], kda.short_conv(last, w)) and y[7:2000].abs().sum() == 0
    H, P, N = 32, 128, 32
    dt = torch.zeros(rows, H, dtype=BF, device="cuda")
    B = torch.randn(300, 1, N, device="cuda").to(BF)
    Bs = torch.zeros(rows, 1, N, dtype=BF, device="cuda")
    Bs[-300:] = B
    A = -torch.ones(H, device="cuda")
    kda.ssm_scan(x.view(rows, H, P), dt, A, Bs, Bs, cu=cu, y=y.view(rows, H, P))
    alone = kda.ssm_scan(last.view(300, H, P), dt[:300], A, B, B)
    torch.cuda.synchronize()
    assert rel_l2(y[-300:].view(300, H, P), _n(alone)) <= 2 * TOL[BF] and y[7:2000].abs().sum() == 0
    # a pool of more than 2^31 elements: 4,300 entries of 32 heads of 128 x 128
    pool = torch.zeros(4300, H, 128, 128, device="cuda")
    xs, ds = torch.randn(2, H, 128, device="cuda").to(BF), torch.zeros(2, H, dtype=BF, device="cuda")
    Bt = torch.randn(2, 1, 128, device="cuda").to(BF)
    got = kda.ssm_step(xs, ds, A, Bt, Bt, pool, slots=_i32([4299, 4290]))
    small = torch.zeros(2, H, 128, 128, device="cuda")
    assert torch.equal(got, kda.ssm_step(xs, ds, A, Bt, Bt, small))
    assert torch.equal(pool[4299], small[0]) and torch.equal(pool[4290], small[1]) and pool[0].abs().sum() == 0


def test_workspace_of_a_named_stream():
    # the helper's own workspace is freed when it returns: what the current stream allocates then must not
    # share it with the call that still runs on the other stream
    ins = _scan_inputs(20000, 2, 128, 128, BF, 5)
    assert kda.kda_ssm_scan_workspace_size(1, 20000, 2, 1, 128, 128, kda.KDA_DTYPE_BF16) > 0
    ref = kda.ssm_scan(*ins)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    ys = []
    for handle in (other, other.cuda_stream) * 4:
        ys.append(kda.ssm_scan(*ins, stream=handle))
        junk = [torch.full((n,), float("nan"), device="cuda") for n in (1 << 18, 1 << 20, 1 << 22)]
        del junk
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref) for y in ys)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_contexts_up_to_the_largest(dtype):
    # positions near 2^31 and beyond it: the same states and outputs, and the snapshots at multiples of page
    H, N, P, T = 2, 64, 64, 300
    x, dt, A, B, C, D, bias = _scan_inputs(T, H, N, P, dtype, 4)
    pool = torch.randn(1, H, N, P, device="cuda")
    want = pool.clone()
    ref = kda.ssm_scan(x, dt, A, B, C, D, bias, state=want, ctx=_i32([123]))  # 123 = (2^31 - 5) % 128
    ctx = 2**31 - 5
    pages, table = torch.zeros(2, H, N, P, device="cuda"), _i32([[0, 1]])
    y = kda.ssm_scan(x, dt, A, B, C, D, bias, state=pool, ctx=_i32([ctx]), block_table=table, pages=pages, page_size=1 << 30)
    torch.cuda.synchronize()
    assert rel_l2(y, _n(ref)) <= TOL[dtype] and rel_l2(pool, _n(want)) <= TOL[F32]
    assert pages[0].abs().sum() == 0 and pages[1].abs().sum() > 0  # 2^31 is the end of block 1
    w = torch.randn(H * P, 4, device="cuda").to(dtype)
    a, b = torch.ones(1, 3, H * P, dtype=dtype, device="cuda"), torch.ones(1, 3, H * P, dtype=dtype, device="cuda")
    ya = kda.short_conv(x.flatten(1), w, state=a, ctx=_i32([2**31 - 1]))
    yb = kda.short_conv(x.flatten(1), w, state=b, ctx=_i32([1]))
    assert torch.equal(ya, yb) and torch.equal(a, b) and kda.kda_get_device_status() == 0


def test_empty_calls():
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")
    none = _i32([])
    assert kda.short_conv(z(0, 64), z(64, 4), cu=_i32([0, 0, 0])).shape == (0, 64)
    assert kda.short_conv(z(2, 0, 64), z(64, 4), head_dim=32, head_major=True).shape == (2, 2, 0, 32)
    assert kda.short_conv_step(z(0, 64), z(64, 4), z(3, 3, 64), slots=none).shape == (0, 64)
    a = torch.ones(2, device="cuda")
    assert kda.ssm_scan(z(0, 2, 16), z(0, 2), a, z(0, 1, 16), z(0, 1, 16)).shape == (0, 2, 16)
    assert kda.ssm_scan(z(3, 0, 2, 16), z(3, 0, 2), a, z(3, 0, 1, 16), z(3, 0, 1, 16)).shape == (3, 0, 2, 16)
    pool = z(1, 2, 16, 16, dtype=F32)
    assert kda.ssm_step(z(0, 2, 16), z(0, 2), a, z(0, 1, 16), z(0, 1, 16), pool, slots=none).shape == (0, 2, 16)
    cu, slots, used = kda.block_map(none, None, none, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), 16, 0)
    torch.cuda.synchronize()
    assert cu.tolist() == [0] and slots.numel() == 0 and used.tolist() == [0] and kda.kda_get_device_status() == 0


def test_short_wait_limit_leaves_results_alone():
    # the scan's waits are bounded by the library's limit; an ordinary call never comes near it
    ins = _scan_inputs(2000, 8, 128, 64, BF, 2)
    ref = kda.ssm_scan(*ins)
    kda.kda_debug_set_wait_limit(200_000_000)
    try:
        y = kda.ssm_scan(*ins)
        assert kda.kda_get_device_status() == 0 and torch.equal(y, ref)
    finally:
        kda.kda_debug_set_wait_limit(0)


def test_stride_of_a_single_row():
    # the stride of one row is never followed, however large (a tensor map would not take it)
    H, N, P = 2, 32, 64
    x, dt, A, B, C, D, bias = _scan_inputs(1, H, N, P, BF, 6)
    ref, y, far = kda.ssm_scan(x, dt, A, B, C, D, bias), torch.empty_like(x), 1 << 42
    code = kda.kda_ssm_scan(x.data_ptr(), far, dt.data_ptr(), far, A.data_ptr(), B.data_ptr(), far, C.data_ptr(), far,
                            D.data_ptr(), bias.data_ptr(), 1, None, 0, None, None, None, None, 0, None, 0, 0, y.data_ptr(),
                            far, 1, 1, H, 1, N, P, 1, None, 0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert code == 0 and rel_l2(y, _n(ref)) <= TOL[BF]
