"""The operators of a layer's cached, packed serving path, as cases that can be timed and compared.

block_map       request lengths -> sequence offsets, block table, token slots
short_conv      short causal convolution of packed prompts (with Swish and the head L2 norm of a KDA layer)
short_conv_step the same for one token of each sequence
ssm_scan        selective state space scan of packed prompts, states in a pool, snapshots at block boundaries
ssm_step        the same for one token of each sequence

`run` computes each in its plain form (elementary torch operations in 32 bits, decays in 64), or, where `own` is
true, by the call that a user makes.  Sizes are this repository's workloads (heads of 128, 16 or 32 of them, 4096 or
8192 tokens, 256 decoded sequences, blocks of 512 tokens) and generic odd ones.
"""
import math
import random

import torch

own = False

EPS = 1e-6
CHUNK = 64  # of the plain scan; blocks are multiples of it


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one decode iteration of a full batch: most requests stay in their last block
        dict(name="map_decode_r256", op="block_map", R=256, rows=256, ctx=8192, page=16, blocks=640),
        # admission of a wave of prompts, long and short ones
        dict(name="map_prompts_r61", op="block_map", R=61, rows=150000, ctx=1000, page=64, blocks=2560),
        # query or key edge of a KDA layer before the prefill kernel: 16 heads of 128, 4096 tokens
        dict(name="conv_qk_h16_t4k", op="short_conv", R=1, rows=4096, C=2048, K=4, dtype="bf16", head_dim=128, norm=True,
             heads=True, ctx=False, packed=False),
        # packed prompts of a hybrid layer (x, B and C of 32 heads of 128 together), some continued from the pool
        dict(name="conv_packed_t64k", op="short_conv", R=8, rows=65536, C=4352, K=4, dtype="bf16", head_dim=0, norm=False,
             heads=False, ctx=True, packed=True),
        # a few short prompts with an odd channel count in 32 bits
        dict(name="conv_f32_odd", op="short_conv", R=5, rows=777, C=515, K=3, dtype="f32", head_dim=0, norm=False,
             heads=False, ctx=True, packed=True),
        # decode of a full batch
        dict(name="conv_step_r256", op="short_conv_step", R=256, C=4352, K=4, dtype="bf16", head_dim=0, norm=False),
        # decode of one sequence: latency
        dict(name="conv_step_r1", op="short_conv_step", R=1, C=2048, K=4, dtype="bf16", head_dim=128, norm=True),
        # one long document
        dict(name="scan_long_t128k", op="ssm_scan", R=1, rows=131072, H=16, G=1, N=128, P=128, dtype="bf16", ctx=False,
             packed=False, page=0),
        # packed prompts, some continued, with a snapshot at every block of 512 tokens
        dict(name="scan_packed_t32k", op="ssm_scan", R=9, rows=32768, H=32, G=2, N=128, P=64, dtype="bf16", ctx=True,
             packed=True, page=512),
        # a short prompt in 32 bits
        dict(name="scan_f32_t300", op="ssm_scan", R=2, rows=600, H=4, G=1, N=64, P=32, dtype="f32", ctx=False, packed=False,
             page=0),
        # decode of a full batch: 256 sequences, 32 heads of 128
        dict(name="step_r256_h32", op="ssm_step", R=256, H=32, G=1, N=128, P=128, dtype="bf16"),
        # decode of one sequence: latency
        dict(name="step_r1_h32", op="ssm_step", R=1, H=32, G=2, N=128, P=64, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["block_map", "short_conv", "short_conv_step", "ssm_scan", "ssm_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "block_map":
        R, page = _log(rng, 1, 700), rng.choice([1, 16, 48, 64, 512])
        rows = R if rng.random() < 0.4 else _log(rng, R, 150000)
        ctx = rng.choice([0, 700, 8192])
        return dict(op=op, R=R, rows=rows, ctx=ctx, page=page, blocks=(ctx + rows) // page + 2)
    if op == "short_conv":
        R, K = _log(rng, 1, 64), rng.choice([2, 3, 4])
        if rng.random() < 0.5:
            H, d = _log(rng, 1, 33), rng.choice([16, 32, 64, 128])
            rows = _log(rng, 1, 30000) * R if R < 3 else R * _log(rng, 1, 900)
            return dict(op=op, R=R, rows=rows, C=H * d, K=K, dtype=dtype, head_dim=d, norm=rng.random() < 0.6,
                        heads=rng.random() < 0.7, ctx=rng.random() < 0.5, packed=False)
        rows = _log(rng, R, 60000)
        C = _log(rng, 1, max(1, min(4352, 250000000 // rows)))
        return dict(op=op, R=R, rows=rows, C=C, K=K, dtype=dtype, head_dim=0, norm=False, heads=False,
                    ctx=rng.random() < 0.5, packed=rows > R)
    if op == "short_conv_step":
        R, K = _log(rng, 1, 512), rng.choice([2, 3, 4])
        if rng.random() < 0.5:
            H, d = _log(rng, 1, 33), rng.choice([16, 32, 64, 128])
            return dict(op=op, R=R, C=H * d, K=K, dtype=dtype, head_dim=d, norm=rng.random() < 0.7)
        return dict(op=op, R=R, C=_log(rng, 1, 4500), K=K, dtype=dtype, head_dim=0, norm=False)
    N, P, G = rng.choice([16, 32, 64, 128, 128]), rng.choice([16, 32, 64, 64, 128]), rng.choice([1, 1, 2, 3])
    H = G * _log(rng, 1, 32 // G)
    if op == "ssm_step":
        return dict(op=op, R=_log(rng, 1, 256), H=H, G=G, N=N, P=P, dtype=dtype)
    R = _log(rng, 1, 40)
    packed = rng.random() < 0.6
    rows = _log(rng, R, 40000 if dtype == "bf16" else 4000)
    rows = rows if packed else max(1, rows // R) * R
    page = rng.choice([0, 128, 512])
    return dict(op=op, R=R, rows=rows, H=H, G=G, N=N, P=P, dtype=dtype, ctx=rng.random() < 0.6, packed=packed, page=page)


def _lens(case):
    """Tokens of each sequence: equal ones, or shares drawn from the sizes alone."""
    R, rows = case["R"], case["rows"]
    if case["op"] != "block_map" and not case["packed"]:
        return [rows // R] * R
    if rows == R:
        return [1] * R
    rng = random.Random(R * 1000003 + rows)
    share = [rng.expovariate(1.0) + 0.05 for _ in range(R)]
    cut, at, lens = sum(share), 0.0, []
    for s in share:
        lo = round(rows * at / cut)
        at += s
        lens.append(round(rows * at / cut) - lo)
    lens[-1] += rows - sum(lens)
    return lens


def _ctx(case):
    """Tokens that each sequence has behind it already; none for about a third of them."""
    rng = random.Random(case["R"] * 7919 + case["rows"])
    most = case["ctx"] if case["op"] == "block_map" else 2000 if case["ctx"] else 0
    return [rng.randint(0, most) if rng.random() < 0.7 else 0 for _ in range(case["R"])]


def _dtype(case):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[case["dtype"]]


# ---- inputs ------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dev = dict(device="cuda")

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, **dev).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, **dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, **dev)

    op, R = case["op"], case["R"]
    s = dict(case=case)
    # every sequence has a place of its own in the pool, in no order
    s["slots"] = torch.randperm(R + 3, generator=gen, **dev)[:R].to(torch.int32)
    if op == "block_map":
        page, blocks = case["page"], case["blocks"]
        lens, ctx = _lens(case), _ctx(case)
        old = [-(-c // page) for c in ctx]
        need = sum(-(-(c + n) // page) - o for c, n, o in zip(ctx, lens, old))
        pages = torch.randperm(sum(old) + need + 64, generator=gen, **dev).to(torch.int32)
        table = torch.full((R, blocks), -1, dtype=torch.int32, **dev)
        old_t = torch.tensor(old, **dev)
        col = torch.arange(blocks, **dev)[None, :]
        first = (torch.cumsum(old_t, 0) - old_t)[:, None]
        held = col < old_t[:, None]
        table = torch.where(held, pages[(first + col).clamp(max=max(0, sum(old) - 1))], table).contiguous()
        # pages are handed out again on every pass over the same state: the table's tail is rewritten, not grown
        s.update(lens=ints(lens), ctx=ints(ctx), table=table, free=pages[sum(old):].clone())
        return s
    t = _dtype(case)
    if op in ("short_conv", "short_conv_step"):
        C, K, rows = case["C"], case["K"], case.get("rows", R)
        # the channels are columns of a wider projection
        wide = normal(rows, C + 16, dtype=t)
        s.update(x=wide[:, :C], w=(normal(C, K) / K ** 0.5).to(t), bias=(0.1 * normal(C)).to(t),
                 state=normal(R + 3, K - 1, C, dtype=t))
    else:
        H, G, N, P, rows = case["H"], case["G"], case["N"], case["P"], case.get("rows", R)
        # x, B and C are columns of the convolution's output
        xbc = normal(rows, H * P + 2 * G * N, dtype=t)
        step = torch.exp(uniform(H) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        s.update(x=xbc[:, :H * P].unflatten(1, (H, P)), B=xbc[:, H * P:H * P + G * N].unflatten(1, (G, N)),
                 C=xbc[:, H * P + G * N:].unflatten(1, (G, N)), dt=normal(rows, H, dtype=t),
                 dt_bias=step + torch.log(-torch.expm1(-step)), A=-(1 + 15 * uniform(H)), D=1 + 0.1 * normal(H),
                 state=0.5 * normal(R + 3, H, N, P))
    if op in ("short_conv", "ssm_scan"):
        lens, ctx = _lens(case), _ctx(case)
        s["T"] = max(lens)
        s["cu"] = ints([sum(lens[:r]) for r in range(R + 1)])
        s["ctx"] = ints(ctx)
        if case.get("page"):
            page = case["page"]
            blocks = max((c + n) // page for c, n in zip(ctx, lens)) + 1
            count = sum((c + n) // page - c // page for c, n in zip(ctx, lens))
            order = torch.randperm(count + 5, generator=gen, **dev).to(torch.int32)
            table = torch.full((R, blocks), -1, dtype=torch.int32)
            at = 0
            for r, (c, n) in enumerate(zip(ctx, lens)):
                k = (c + n) // page - c // page
                table[r, c // page:c // page + k] = torch.arange(at, at + k, dtype=torch.int32)
                at += k
            table = table.cuda()
            s["table"] = torch.where(table >= 0, order[table.clamp(min=0).long()], table).contiguous()
            s["pages"] = torch.zeros(count + 5, case["H"], case["N"], case["P"], **dev)
    return s


# ---- plain forms ---------------------------------------------------------------

def _plain_map(s):
    case, lens, ctx = s["case"], s["lens"].long(), s["ctx"].long()
    page, R, rows = case["page"], case["R"], case["rows"]
    cu = torch.zeros(R + 1, dtype=torch.int64, device=lens.device)
    cu[1:] = torch.cumsum(lens, 0)
    old = (ctx + page - 1) // page
    new = (ctx + lens + page - 1) // page - old
    first = torch.cumsum(new, 0) - new
    col = torch.arange(case["blocks"], device=lens.device)[None, :]
    fresh = (col >= old[:, None]) & (col < (old + new)[:, None])
    at = (first[:, None] + col - old[:, None]).clamp(0, s["free"].numel() - 1)
    s["table"].copy_(torch.where(fresh, s["free"][at], s["table"]))
    tok = torch.arange(rows, device=lens.device)
    r = torch.searchsorted(cu[1:], tok, right=True).clamp(max=R - 1)
    pos = ctx[r] + tok - cu[r]
    slot = s["table"][r, pos // page].long() * page + pos % page
    return dict(cu=cu.to(torch.int32), table=s["table"], slots=slot, used=new.sum().to(torch.int32).reshape(1))


def _history(s, carried):
    """[rows, K, C] in 32 bits: the K inputs that each row's convolution sees, oldest first."""
    x, K = s["x"].float(), s["case"]["K"]
    rows, cu = x.shape[0], s["cu"].long()
    row = torch.arange(rows, device=x.device)
    r = torch.searchsorted(cu[1:], row, right=True)
    src = row[:, None] - (K - 1) + torch.arange(K, device=x.device)[None, :]
    back = src - cu[r][:, None]  # position in the sequence; negative: in its pool entry
    old = s["state"].float()[s["slots"].long()[r]]  # [rows, K-1, C]
    old = torch.where(carried[r][:, None, None], old, torch.zeros_like(old))
    old = old.gather(1, (back + K - 1).clamp(0, K - 2)[:, :, None].expand(-1, -1, x.shape[1]))
    return torch.where((back >= 0)[:, :, None], x[src.clamp(min=0)], old)


def _edge(s, v):
    """Swish and the optional L2 norm of each head."""
    case = s["case"]
    v = v / (1 + torch.exp(-v))
    if case["norm"]:
        h = v.unflatten(1, (-1, case["head_dim"]))
        v = (h / torch.sqrt((h * h).sum(2, keepdim=True) + EPS)).flatten(1)
    return v


def _plain_conv(s):
    case, K = s["case"], s["case"]["K"]
    hist = _history(s, s["ctx"] > 0)
    y = _edge(s, (hist * s["w"].float().t()[None]).sum(1) + s["bias"].float()).to(s["x"].dtype)
    # the pool keeps the last K - 1 inputs of each sequence that has any
    cu = s["cu"].long()
    some = cu[1:] > cu[:-1]
    last = hist[(cu[1:] - 1).clamp(min=0), 1:].to(s["state"].dtype)
    at = s["slots"].long()
    s["state"][at] = torch.where(some[:, None, None], last, s["state"][at])
    if case["heads"]:
        y = y.view(case["R"], -1, case["C"] // case["head_dim"], case["head_dim"]).transpose(1, 2).contiguous()
    return dict(y=y, state=s["state"])


def _plain_conv_step(s):
    at = s["slots"].long()
    hist = torch.cat([s["state"][at].float(), s["x"].float()[:, None]], 1)
    y = _edge(s, (hist * s["w"].float().t()[None]).sum(1) + s["bias"].float()).to(s["x"].dtype)
    s["state"][at] = hist[:, 1:].to(s["state"].dtype)
    return dict(y=y, state=s["state"])


def _delta(s):
    v = s["dt"].double() + s["dt_bias"].double()
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _plain_step(s):
    at, H, G = s["slots"].long(), s["case"]["H"], s["case"]["G"]
    delta = _delta(s)
    B, C = (s[k].float().repeat_interleave(H // G, 1) for k in ("B", "C"))
    x = s["x"].float()
    keep = torch.exp(delta * s["A"].double()).float()
    S = s["state"][at] * keep[:, :, None, None] + (B * delta.float()[:, :, None])[:, :, :, None] * x[:, :, None, :]
    s["state"][at] = S
    y = (S * C[:, :, :, None]).sum(2) + s["D"][None, :, None] * x
    return dict(y=y.to(s["x"].dtype), state=s["state"])


def _plain_scan(s):
    """Chunks of 64 tokens that end at multiples of 64 of the sequence's position: products inside a chunk, and one
    product over the chunks' states with the decays between them."""
    case, Q = s["case"], CHUNK
    R, H, G, N, P = case["R"], case["H"], case["G"], case["N"], case["P"]
    cu, ctx, at = s["cu"].long(), s["ctx"].long(), s["slots"].long()
    dev = cu.device
    off = ctx % Q
    nc = -(-(s["T"] + Q - 1) // Q)
    local = torch.arange(nc * Q, device=dev)[None, :] - off[:, None]
    ok = (local >= 0) & (local < (cu[1:] - cu[:-1])[:, None])
    row = (cu[:-1, None] + local).clamp(0, case["rows"] - 1)

    def padded(t):
        t = t[row]
        return torch.where(ok.reshape(ok.shape + (1,) * (t.dim() - 2)), t, torch.zeros_like(t)).unflatten(1, (nc, Q))

    x, B, C = (padded(s[k]).float() for k in ("x", "B", "C"))
    x = x.unflatten(3, (G, H // G))
    delta = padded(_delta(s)).unflatten(3, (G, H // G))  # [R, nc, Q, G, h]
    A = s["A"].double().view(G, H // G)
    cs = torch.cumsum(delta * A, 2)
    d32 = delta.float()
    tri = torch.ones(Q, Q, dtype=torch.bool, device=dev).tril()[:, :, None, None]
    between = torch.exp(torch.where(tri, cs[:, :, :, None] - cs[:, :, None], -math.inf)).float()  # [R, nc, t, s, G, h]
    gram = torch.einsum("rctgn,rcsgn->rctsg", C, B)
    w = gram[..., None] * between * d32[:, :, None]
    y = torch.einsum("rctsgh,rcsghp->rctghp", w, x)
    del between, w
    own_part = torch.einsum("rcsgn,rcsghp->rcghnp", B, x * (d32 * torch.exp(cs[:, :, -1:] - cs).float())[..., None])
    # states at the chunks' starts and after the last: products with the decay from each chunk's end
    start = torch.where((ctx > 0)[:, None, None, None], s["state"][at], 0.0).view(R, 1, G, H // G, N, P)
    parts = torch.cat([start, own_part], 1).flatten(4)  # [R, nc + 1, G, h, N P]
    total = torch.cumsum(torch.cat([torch.zeros_like(cs[:, :1, -1]), cs[:, :, -1]], 1), 1)  # [R, nc + 1, G, h]
    tri = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=dev).tril()[:, :, None, None]
    far = torch.exp(torch.where(tri, total[:, :, None] - total[:, None], -math.inf)).float()  # [R, c, c', G, h]
    states = torch.einsum("rcdgh,rdghm->rcghm", far, parts).unflatten(4, (N, P))
    y = y + torch.exp(cs).float()[..., None] * torch.einsum("rctgn,rcghnp->rctghp", C, states[:, :-1])
    y = (y + s["D"].view(G, H // G, 1) * x).flatten(3, 4).flatten(1, 2)[ok].to(s["x"].dtype)
    s["state"][at] = torch.where((cu[1:] > cu[:-1])[:, None, None, None], states[:, -1].flatten(1, 2), s["state"][at])
    if not case["page"]:
        return dict(y=y, state=s["state"])
    # states[r, c] is the state at position ctx - off + c Q
    pos = (ctx - off)[:, None] + torch.arange(nc + 1, device=dev)[None, :] * Q
    hit = (pos % case["page"] == 0) & (pos > ctx[:, None]) & (pos <= (ctx + cu[1:] - cu[:-1])[:, None])
    r, c = hit.nonzero(as_tuple=True)
    s["pages"][s["table"][r, pos[r, c] // case["page"] - 1].long()] = states[r, c].flatten(1, 2)
    return dict(y=y, state=s["state"], pages=s["pages"])


# ---- one pass --------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"block_map": _plain_map, "short_conv": _plain_conv, "short_conv_step": _plain_conv_step,
                "ssm_scan": _plain_scan, "ssm_step": _plain_step}[op](s)
    from gated_delta_rule_117_b200 import kda
    case = s["case"]
    if op == "block_map":
        cu, slots, used = kda.block_map(s["lens"], s["ctx"], s["free"], s["table"], case["page"], case["rows"])
        return dict(cu=cu, table=s["table"], slots=slots, used=used)
    if op == "short_conv":
        x = s["x"] if case["packed"] else s["x"].unflatten(0, (case["R"], -1))
        y = kda.short_conv(x, s["w"], s["bias"], state=s["state"], slots=s["slots"], ctx=s["ctx"],
                           cu=s["cu"] if case["packed"] else None, head_dim=case["head_dim"], l2norm=case["norm"],
                           head_major=case["heads"], eps=EPS)
        return dict(y=y if case["heads"] else y.view(case["rows"], -1), state=s["state"])
    if op == "short_conv_step":
        y = kda.short_conv_step(s["x"], s["w"], s["state"], s["bias"], slots=s["slots"], head_dim=case["head_dim"],
                                l2norm=case["norm"], eps=EPS)
        return dict(y=y, state=s["state"])
    if op == "ssm_step":
        y = kda.ssm_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], s["D"], s["dt_bias"], slots=s["slots"])
        return dict(y=y, state=s["state"])
    x, dt, B, C = (s[k] if case["packed"] else s[k].unflatten(0, (case["R"], -1)) for k in ("x", "dt", "B", "C"))
    more = dict(block_table=s["table"], pages=s["pages"], page_size=case["page"]) if case["page"] else {}
    y = kda.ssm_scan(x, dt, s["A"], B, C, s["D"], s["dt_bias"], state=s["state"], slots=s["slots"], ctx=s["ctx"],
                     cu=s["cu"] if case["packed"] else None, **more)
    out = dict(y=y.view(case["rows"], case["H"], case["P"]), state=s["state"])
    if case["page"]:
        out["pages"] = s["pages"]
    return out


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    op, R = case["op"], case["R"]
    e = 2 if case.get("dtype") == "bf16" else 4
    if op == "block_map":
        lens, ctx = _lens(case), _ctx(case)
        new = sum(-(-(c + n) // case["page"]) - -(-c // case["page"]) for c, n in zip(ctx, lens))
        # a token's slot needs the entry of its block in the table
        held = sum(1 for c, n in zip(ctx, lens) if n and c % case["page"])
        return dict(bytes=8 * R + 4 * (R + 2) + 8 * case["rows"] + 8 * new + 4 * held, flops=0)
    if op == "short_conv":
        lens, ctx, C, K = _lens(case), _ctx(case), case["C"], case["K"]
        state = sum((2 if c else 1) for n, c in zip(lens, ctx) if n) * (K - 1) * C * e
        return dict(bytes=2 * case["rows"] * C * e + state + C * (K + 1) * e + 12 * R, flops=case["rows"] * C * (2 * K + 4))
    if op == "short_conv_step":
        C, K = case["C"], case["K"]
        return dict(bytes=2 * R * C * e + 2 * R * (K - 1) * C * e + C * (K + 1) * e + 4 * R, flops=R * C * (2 * K + 4))
    H, G, N, P = case["H"], case["G"], case["N"], case["P"]
    if op == "ssm_step":
        return dict(bytes=8 * R * H * N * P + R * e * (2 * H * P + 2 * G * N + H) + 12 * H + 4 * R, flops=R * H * N * P * 5)
    lens, ctx = _lens(case), _ctx(case)
    states = sum((2 if c else 1) for n, c in zip(lens, ctx) if n)
    if case["page"]:
        states += sum((c + n) // case["page"] - c // case["page"] for c, n in zip(ctx, lens))
    rows = case["rows"]
    # the fewest operations are the recurrence's own: decay, write and read of each entry of the state
    return dict(bytes=rows * e * (2 * H * P + 2 * G * N + H) + 4 * states * H * N * P + 12 * H + 12 * R,
                flops=rows * H * N * P * 5)


# ---- in 64 bits --------------------------------------------------------------------

def exact(case, seed):
    """From the definitions: tokens one after the other."""
    s = prepare(case, seed)
    op, R = case["op"], case["R"]
    if op == "block_map":
        return None
    at = s["slots"].long()
    if op in ("short_conv", "short_conv_step"):
        C, K, d = case["C"], case["K"], case["head_dim"]
        lens = _lens(case) if op == "short_conv" else [1] * R
        ctx = _ctx(case) if op == "short_conv" else [1] * R
        x, w, b, pool = (s[k].double() for k in ("x", "w", "bias", "state"))
        kept, parts, lo = pool.clone(), [], 0
        for r in range(R):
            n = lens[r]
            before = pool[at[r]] if ctx[r] else torch.zeros_like(pool[0])
            seq = torch.cat([before, x[lo:lo + n]])
            lo += n
            v = b.repeat(n, 1)
            for k in range(K):
                v = v + seq[k:k + n] * w[:, k]
            v = v * torch.sigmoid(v)
            if case["norm"]:
                v = v.view(n, C // d, d)
                v = (v / (v.square().sum(-1, keepdim=True) + EPS).sqrt()).view(n, C)
            parts.append(v)
            if n:
                kept[at[r]] = seq[n:]
        y = torch.cat(parts)
        if case.get("heads"):
            y = torch.stack([p.view(-1, C // d, d).permute(1, 0, 2) for p in parts])
        return dict(y=y, state=kept)
    H, G, N, P = case["H"], case["G"], case["N"], case["P"]
    lens = _lens(case) if op == "ssm_scan" else [1] * R
    ctx = _ctx(case) if op == "ssm_scan" else [1] * R
    page = case.get("page", 0)
    dev = at.device
    n, c = torch.tensor(lens, device=dev), torch.tensor(ctx, device=dev)
    first = torch.cumsum(n, 0) - n
    pool = s["state"].double()
    S = torch.where((c > 0)[:, None, None, None], pool[at], 0.0)
    A, bias, D = s["A"].double(), s["dt_bias"].double(), s["D"].double()
    y = torch.empty(s["x"].shape, dtype=torch.float64, device=dev)
    pages = s["pages"].double() if page else None
    # the longest first: the sequences that still have a token are the first ones
    order = torch.argsort(n, descending=True, stable=True)
    S, by_len = S[order], sorted(lens, reverse=True)
    live = R
    for t in range(by_len[0]):
        while live and by_len[live - 1] <= t:
            live -= 1
        who = order[:live]
        row = first[who] + t
        step = torch.nn.functional.softplus(s["dt"][row].double() + bias, threshold=1e9)
        x = s["x"][row].double()
        B, C = (s[k][row].double().repeat_interleave(H // G, 1) for k in ("B", "C"))
        cur = S[:live]
        cur.mul_(torch.exp(step * A)[:, :, None, None]).add_((B * step[:, :, None])[..., None] * x[:, :, None])
        y[row] = (C[:, :, None] @ cur)[:, :, 0] + D[:, None] * x
        if page:
            for i, r in enumerate(order[:live].tolist() if any((k + t + 1) % page == 0 for k in ctx) else []):
                if (ctx[r] + t + 1) % page == 0:
                    pages[s["table"][r, (ctx[r] + t) // page].long()] = cur[i]
    pool[at[order]] = torch.where((n[order] > 0)[:, None, None, None], S, pool[at[order]])
    return dict(y=y, state=pool, pages=pages) if page else dict(y=y, state=pool)
