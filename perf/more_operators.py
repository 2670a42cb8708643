"""Measured cases of the 4-bit caches and of moves within a pool: attention
over caches of E2M1 codes with a scale a token, tokens written into a cache and
read back, finished steps committed between 4-bit caches, blocks copied and
compacted within their pools.

With ``own`` false the operators run in their plain form (elementary torch
operations, 32 bits or more whatever the storage type); with ``own`` true they
run through the library's entry points.
"""
import math

import torch

own = False

F32, BF16, FP8, FP4 = "f32", "bf16", "fp8", "fp4"
TORCH = {F32: torch.float32, BF16: torch.bfloat16, FP8: torch.float8_e4m3fn, FP4: torch.uint8}
# bytes of a cached token's key (or value) of 128 elements, with its half of the scales
ROW = {F32: 512, BF16: 256, FP8: 128, FP4: 66}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _decode(name, problems, workers, chunk, hq, hkv, common, block, ragged=False, append=False, theta=1e6):
    return {"name": name, "op": "decode", "problems": problems, "workers": workers, "chunk": chunk, "hq": hq,
            "hkv": hkv, "common": common, "block": block, "ragged": ragged, "append": append, "theta": theta}


def _write(name, dtype, layers, rows, tokens, hkv, d, theta=1e6):
    return {"name": name, "op": "write", "dtype": dtype, "layers": layers, "rows": rows, "tokens": tokens, "hkv": hkv,
            "d": d, "theta": theta}


def _commit(name, layers, hkv, steps, tokens, history, theta=1e6):
    return {"name": name, "op": "commit", "layers": layers, "hkv": hkv, "steps": steps, "tokens": tokens,
            "history": history, "theta": theta}


def _move(name, dtype, kind, layers, hkv, d, blocks, block):
    return {"name": name, "op": "move", "dtype": dtype, "kind": kind, "layers": layers, "hkv": hkv, "d": d,
            "blocks": blocks, "block": block}


def listed():
    return [
        # two workers behind a short prompt: latency
        _decode("decode4-short", 1, 2, 0, 40, 8, 1001, 250),
        # four workers on a 16K history: the ordinary step
        _decode("decode4-history-16k", 1, 4, 0, 40, 8, 16384, 512),
        # the same with each worker's new token written by the call
        _decode("decode4-append-16k", 1, 4, 0, 40, 8, 16384, 512, append=True),
        # query chunks of two tokens a worker on a 32K history
        _decode("decode4-chunk-32k", 1, 4, 2, 32, 8, 32768, 1024),
        # a batch of independent problems of unlike lengths
        _decode("decode4-serve-ragged", 8, 4, 0, 40, 8, 65536, 2048, ragged=True),
        # a step's tokens of four workers into a 16-bit cache: latency
        _write("write-step-bf16", BF16, 1, 4, 1, 8, 128),
        # a prompt of odd length into an 8-bit cache
        _write("write-prompt-fp8", FP8, 1, 1, 5003, 8, 128),
        # long prompts into a 4-bit cache, read back
        _write("write-prompt-fp4", FP4, 4, 2, 16384, 8, 128),
        # a finished step's tokens, a few layers
        _commit("commit4-step", 4, 8, 1, 37, 1001),
        # the finished steps of four workers in all layers of a model
        _commit("commit4-model", 36, 8, 4, 1024, 4096),
        # a worker's step forked for three others, in all layers
        _move("fork-bf16", BF16, "fork", 64, 8, 128, 3, 512),
        # the blocks left between finished ones slide down, in all layers
        _move("compact-fp8", FP8, "compact", 36, 8, 128, 16, 1024),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "write", "write", "commit", "move"])
    if op == "decode":
        hq, hkv = rng.choice([(40, 8), (32, 8), (4, 2), (8, 8), (16, 1)])
        problems, workers = rng.choice([1, 1, 1, 2, 5, 8]), rng.choice([1, 2, 3, 4, 6])
        append = rng.random() < 0.25
        chunk = 0 if append else rng.choice([0, 0, 1, 2, 3])
        block = max(_spread(rng, 1, 2048), chunk)
        common = _spread(rng, 1, 65536)
        rows = problems * workers * max(1, chunk)
        common = max(1, min(common, int(1.5e7 / (rows * hkv)) - workers * block, int(8e7 / (rows * hq)) - workers * block))
        c = _decode("", problems, workers, chunk, hq, hkv, common, block, rng.random() < 0.5, append,
                    rng.choice([1e4, 1e6]))
    elif op == "write":
        dtype = rng.choice([F32, BF16, FP8, FP4, FP4])
        layers, rows, hkv = _spread(rng, 1, 16), rng.choice([1, 2, 4, 7]), rng.choice([1, 2, 8])
        tokens = min(_spread(rng, 1, 20000), max(1, 1000000 // (layers * rows * hkv)))
        c = _write("", dtype, layers, rows, tokens, hkv, rng.choice([64, 128]) if dtype in (F32, BF16) else 128,
                   rng.choice([1e4, 1e6]))
    elif op == "commit":
        layers, hkv, steps = _spread(rng, 1, 36), rng.choice([1, 2, 8]), rng.choice([1, 2, 4])
        c = _commit("", layers, hkv, steps, _spread(rng, 1, 1024), _spread(rng, 1, 4096), rng.choice([1e4, 1e6]))
    else:
        dtype = rng.choice([F32, BF16, FP8, FP4])
        c = _move("", dtype, rng.choice(["fork", "compact"]), _spread(rng, 1, 36), rng.choice([1, 2, 8]),
                  rng.choice([64, 128]) if dtype in (F32, BF16) else 128, rng.choice([1, 2, 3, 5, 8]),
                  _spread(rng, 1, 512))
    del c["name"]
    return c


# --------------------------------------------------------------------------
# the 4-bit format
# --------------------------------------------------------------------------

# E2M1: code 0 .. 7 is a magnitude, 8 more the sign; two to a byte, the even
# element in the low bits.  A token's keys (and its values) of one kv head
# share a scale in bf16: their largest magnitude over 6.
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# borders between neighbouring magnitudes; at a border the even code stands
BORDERS = ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0))


def _encode(x):
    """x [..., D] fp32 -> codes [..., D] (int64), scales [...] (bf16).  Tokens
    below 2^-100 are zero, tokens of 2^100 or more (or not finite) NaN."""
    a = x.abs()
    top = a.amax(-1)
    scale = (top / 6.0).to(torch.bfloat16).float()
    scale = torch.where(scale < 2.0 ** -100, 0.0, scale)
    scale = torch.where(top < 2.0 ** 100, scale, math.nan)
    s = scale[..., None]
    # a border times a scale is exact in 32 bits, so nothing is divided
    code = torch.zeros(x.shape, dtype=torch.uint8, device=x.device)
    (b0, _), (b1, _), (b2, _), (b3, _), (b4, _), (b5, _), (b6, _) = BORDERS
    code += (a > b0 * s).byte() + (a >= b1 * s).byte() + (a > b2 * s).byte() + (a >= b3 * s).byte()
    code += (a > b4 * s).byte() + (a >= b5 * s).byte() + (a > b6 * s).byte()
    code = torch.where(s > 0, code + 8 * (x < 0).byte(), 0).byte()
    return code, scale.to(torch.bfloat16)


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _values(codes, scale):
    """Values of packed codes [..., D / 2] under scales [...], fp32."""
    lut = torch.tensor([*LEVELS, *(-x for x in LEVELS)], device=codes.device)
    v = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2)
    return v * scale.float()[..., None]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _layout(case, g):
    """Host lists: block lengths and starts, the rows' views and what they see."""
    P, W, T = case["problems"], case["workers"], case["chunk"]
    lens, starts, at = [], [], 0
    for p in range(P):
        row = [case["common"]] + [max(1, T, case["block"] * (W - w) // W) for w in range(W)]
        if case["ragged"]:
            row = [int(torch.randint(max(1, T, n // 4), n + 1, (1,), generator=g)) for n in row]
        for n in row:
            lens.append(n)
            starts.append(at)
            at += n
    views, offs, limits, q_pos, own_block = [], [], [], [], []
    for p in range(P):
        base = p * (W + 1)
        for w in range(W):
            mine = base + 1 + w
            order = [base] + [base + 1 + o for o in range(W) if o != w] + [mine]
            off = [0]
            for b in order:
                off.append(off[-1] + lens[b])
            total = off.pop()
            for t in range(max(1, T)):
                views.append(order)
                offs.append(off)
                limits.append([-1] * W + [lens[mine] - T + t + 1 if T else -1])
                # behind the view, or the token's own place in it
                q_pos.append(total - T + t if T else total - 1 if case["append"] else total)
                own_block.append(mine)
    capacity = P * (case["common"] + sum(max(1, T, case["block"] * (W - w) // W) for w in range(W)))
    return dict(lens=lens, starts=starts, views=views, offs=offs, limits=limits, q_pos=q_pos, own_block=own_block,
                capacity=capacity)


def _prepare_decode(case, seed):
    g = torch.Generator().manual_seed(seed)
    L = _layout(case, g)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    W, hq, hkv, d = case["workers"], case["hq"], case["hkv"], 128
    R, n_view = len(L["views"]), W + 1
    s = {"case": case, "layout": L}
    pools, scales = [], []
    for which in range(2):
        x = torch.randn(hkv, L["capacity"], d, generator=gd, device="cuda")
        # tokens of unlike size, as a model's are; the first key of a history draws attention
        x *= torch.exp(0.3 * torch.randn(hkv, L["capacity"], 1, generator=gd, device="cuda"))
        if which == 0:
            for p in range(case["problems"]):
                x[:, L["starts"][p * n_view]] *= 8.0
        code, scale = _encode(x)
        pools.append(_pack(code))
        scales.append(scale)
        del x, code
    s["k_cache"], s["v_cache"], s["kv_scale"] = pools[0], pools[1], torch.stack(scales, -1)
    s["q"] = torch.randn(R, hq, d, generator=gd, device="cuda").to(torch.bfloat16)
    s["out"] = torch.zeros_like(s["q"])
    if case["append"]:  # every row's new token is the last one of its own block
        s["k_new"] = torch.randn(R, hkv, d, generator=gd, device="cuda").to(torch.bfloat16)
        s["v_new"] = torch.randn(R, hkv, d, generator=gd, device="cuda").to(torch.bfloat16)
        s["at"] = _int([L["lens"][b] - 1 for b in L["own_block"]])
        s["slot"] = _int([L["starts"][b] + L["lens"][b] - 1 for b in L["own_block"]])
    # what the plain form indexes with: the view's tokens (padded), their entries, what a row sees of them
    longest = max(sum(L["lens"][b] for b in view) for view in L["views"])
    lens = _int([[L["lens"][b] for b in view] for view in L["views"]]).long()
    starts = _int([[L["starts"][b] for b in view] for view in L["views"]]).long()
    limit = _int(L["limits"]).long()
    at = torch.arange(longest, device="cuda").expand(R, longest)
    ends = lens.cumsum(1)
    ent = torch.searchsorted(ends, at.contiguous(), right=True).clamp(max=n_view - 1)
    within = at - (ends - lens).gather(1, ent)
    seen = at < ends[:, -1:]
    s["token"] = torch.where(seen, starts.gather(1, ent) + within, 0)
    limit = torch.where(limit < 0, lens, limit).gather(1, ent)
    s["seen"] = seen & (within < limit)
    s["shift"] = torch.where(seen, _int(L["offs"]).long().gather(1, ent), 0)
    s["position"] = _int(L["q_pos"]).long()
    if own:
        from concurrent_shared_kv_gb300 import engine
        t = engine.DecodeSession(n_rows=R, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, n_blocks=len(L["lens"]),
                                 max_view_blocks=n_view, capacity=L["capacity"], dtype=torch.bfloat16,
                                 rope_theta=case["theta"], kv_fp4=True, view_limits=case["chunk"] > 0)
        t.set_metadata(L["starts"], L["lens"], L["views"], L["offs"], L["q_pos"])
        if case["chunk"]:
            t.plan_limited(L["limits"])
        elif case["append"]:
            t.plan_append(L["own_block"], s["at"])
        else:
            t.plan()
        s["session"] = t
    return s


def _prepare_write(case, seed):
    gd = torch.Generator(device="cuda").manual_seed(seed)
    g = torch.Generator().manual_seed(seed)
    layers, rows, n, hkv, d = case["layers"], case["rows"], case["tokens"], case["hkv"], case["d"]
    dtype = case["dtype"]
    act = torch.float32 if dtype == F32 else torch.bfloat16
    s = {"case": case}
    # each row's tokens stand behind what its block holds already
    held = torch.randint(0, 1 + n // 4, (rows,), generator=g)
    if n == 1:
        held = torch.randint(0, 600, (rows,), generator=g)
    capacity = rows * ((600 if n == 1 else n // 4) + n)
    start = torch.cat([torch.zeros(1, dtype=torch.int64), (held + n).cumsum(0)])[:rows]
    pos = held[:, None] + torch.arange(n)
    s["pos"] = pos.reshape(-1).int().cuda()
    s["slot"] = (start[:, None] + pos).reshape(-1).int().cuda()
    shape = (layers, rows * n, hkv, d)
    size = torch.exp(0.3 * torch.randn(shape[:-1], generator=gd, device="cuda"))[..., None]
    s["k_new"] = (torch.randn(shape, generator=gd, device="cuda") * size).to(act)
    s["v_new"] = torch.randn(shape, generator=gd, device="cuda").to(act)
    width = d // 2 if dtype == FP4 else d
    s["k_cache"] = torch.zeros(layers, hkv, capacity, width, dtype=torch.uint8 if dtype in (FP8, FP4) else act,
                               device="cuda")
    s["v_cache"] = torch.zeros_like(s["k_cache"])
    if dtype == FP8:
        s["k_cache"], s["v_cache"] = s["k_cache"].view(torch.float8_e4m3fn), s["v_cache"].view(torch.float8_e4m3fn)
        s["k_scale"] = s["k_new"].float().abs().amax(dim=(1, 3)) / 448.0  # [layers, Hkv]
        s["v_scale"] = s["v_new"].float().abs().amax(dim=(1, 3)) / 448.0
    if dtype == FP4:
        s["kv_scale"] = torch.zeros(layers, hkv, capacity, 2, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros(shape, dtype=act, device="cuda")
        s["v_out"] = torch.zeros(shape, dtype=act, device="cuda")
    return s


def _codes_of(gd, layers, hkv, tokens):
    """4-bit pools of `tokens` tokens: packed keys and values, scales."""
    k, v = torch.empty(2, layers, hkv, tokens, 64, dtype=torch.uint8, device="cuda")
    scale = torch.empty(layers, hkv, tokens, 2, dtype=torch.bfloat16, device="cuda")
    for l in range(layers):
        for i, pool in enumerate((k, v)):
            code, scale[l, :, :, i] = _encode(torch.randn(hkv, tokens, 128, generator=gd, device="cuda"))
            pool[l] = _pack(code)
    return k, v, scale


def _prepare_commit(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    layers, hkv, steps, n, history = case["layers"], case["hkv"], case["steps"], case["tokens"], case["history"]
    s = {"case": case}
    lens = [int(torch.randint(max(1, n // 2), n + 1, (1,), generator=g)) for _ in range(steps)] if steps > 1 else [n]
    # the steps stand in the workers' pool; behind the history there is room for them
    s["k_src"], s["v_src"], s["scale_src"] = _codes_of(gd, layers, hkv, steps * n)
    room = history + steps * n
    s["k_dst"], s["v_dst"] = torch.zeros(2, layers, hkv, room, 64, dtype=torch.uint8, device="cuda")
    s["scale_dst"] = torch.zeros(layers, hkv, room, 2, dtype=torch.bfloat16, device="cuda")
    dst, at = [], history
    for m in lens:
        dst.append(at)
        at += m
    s["begin"], s["lens"], s["to"] = [i * n for i in range(steps)], lens, dst
    # keys stand at positions in their own block; in the history they stand at dst
    s["src"] = torch.cat([torch.arange(b, b + m) for b, m in zip(s["begin"], lens)]).cuda()
    s["dst"] = torch.cat([torch.arange(b, b + m) for b, m in zip(dst, lens)]).cuda()
    s["delta"] = torch.cat([torch.full((m,), b) for b, m in zip(dst, lens)]).cuda()
    s["slot"] = torch.arange(history, room, dtype=torch.int32, device="cuda")  # what is read back
    s["k_out"], s["v_out"] = torch.zeros(2, layers, steps * n, hkv, 128, dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_move(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    layers, hkv, d, n, most = case["layers"], case["hkv"], case["d"], case["blocks"], case["block"]
    draw_len = lambda: int(torch.randint(max(1, most // 2), most + 1, (1,), generator=g))  # noqa: E731
    s = {"case": case}
    if case["kind"] == "fork":  # one block copied to n places of its own behind it
        m = most
        begin, lens, to = [5] * n, [m] * n, [5 + m + 3 + i * (m + 7) for i in range(n)]
    else:  # n blocks with gaps between them, each moved down to the one before
        begin, lens, to, at, down = [], [], [], 0, 0
        for _ in range(n):
            at += draw_len()  # a freed block
            m = draw_len()
            begin.append(at)
            lens.append(m)
            to.append(down)
            at += m
            down += m
    capacity = 2 * n * most if case["kind"] == "compact" else 5 + most + n * (most + 7)
    s["begin"], s["lens"], s["to"] = begin, lens, to
    s["src"] = torch.cat([torch.arange(b, b + m) for b, m in zip(begin, lens)]).cuda()
    s["dst"] = torch.cat([torch.arange(b, b + m) for b, m in zip(to, lens)]).cuda()
    if case["dtype"] == FP4:
        s["k_cache"], s["v_cache"], s["kv_scale"] = _codes_of(gd, layers, hkv, capacity)
        s["slot"] = torch.arange(capacity, dtype=torch.int32, device="cuda")  # what is read back
        s["k_out"], s["v_out"] = torch.zeros(2, layers, capacity, hkv, 128, dtype=torch.bfloat16, device="cuda")
    else:
        dt = TORCH[case["dtype"]]
        s["k_cache"], s["v_cache"] = (torch.empty(layers, hkv, capacity, d, dtype=dt, device="cuda") for _ in range(2))
        for l in range(layers):
            for c in (s["k_cache"], s["v_cache"]):
                c[l] = torch.randn(hkv, capacity, d, generator=gd, device="cuda").to(dt)
    return s


def prepare(case, seed):
    return {"decode": _prepare_decode, "write": _prepare_write, "commit": _prepare_commit,
            "move": _prepare_move}[case["op"]](case, seed)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _rotate(x, position, theta):
    """x [..., D] rotated at `position` (integers, broadcast over x's leading
    dimensions): element i pairs with i + D/2; the angle in 64 bits."""
    half = x.shape[-1] // 2
    freq = theta ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    angle = position[..., None].double() * freq
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _read_plain(s, k, v, scale):
    """The tokens `slot` of 4-bit pools [layers][Hkv][cap] into k_out, v_out."""
    at = s["slot"].long()
    for_k = _values(k[:, :, at], scale[:, :, at, 0])
    s["k_out"].copy_(for_k.transpose(1, 2))
    s["v_out"].copy_(_values(v[:, :, at], scale[:, :, at, 1]).transpose(1, 2))
    return s["k_out"], s["v_out"]


def _read_own(s, k, v, scale):
    from concurrent_shared_kv_gb300 import engine
    return engine.cache_read(s["slot"], k, v, kv_scale=scale, k_out=s["k_out"], v_out=s["v_out"])


def _run_decode_plain(s):
    case, theta = s["case"], s["case"]["theta"]
    hq, hkv, d = case["hq"], case["hkv"], 128
    R = s["q"].shape[0]
    new = []
    if case["append"]:
        slot = s["slot"].long()
        for i, x in enumerate((_rotate(s["k_new"], s["at"][:, None], theta), s["v_new"].float())):
            code, scale = _encode(x)  # [R, Hkv, D]
            packed, scale = _pack(code).transpose(0, 1), scale.transpose(0, 1)
            s["v_cache" if i else "k_cache"][:, slot] = packed
            s["kv_scale"][:, slot, i] = scale
            new.append(_values(packed, scale).transpose(0, 1).to(torch.bfloat16))
    k = _values(s["k_cache"], s["kv_scale"][..., 0])[:, s["token"]].transpose(0, 1)  # [R, Hkv, L, D]
    k = _rotate(k, s["shift"][:, None], theta)
    q = _rotate(s["q"], s["position"][:, None], theta).reshape(R, hkv, hq // hkv, d)
    score = q @ k.transpose(2, 3) * d ** -0.5
    del k
    score = score.masked_fill(~s["seen"][:, None, None], -math.inf)
    e = (score - score.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    v = _values(s["v_cache"], s["kv_scale"][..., 1])[:, s["token"]].transpose(0, 1)
    s["out"].copy_((e @ v / e.sum(-1, keepdim=True)).reshape(R, hq, d))
    return (s["out"], *new)


def _run_decode_own(s):
    t = s["session"]
    if s["case"]["append"]:
        from concurrent_shared_kv_gb300 import engine
        t.append_decode_planned_fp4(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["kv_scale"],
                                    out=s["out"], want_lse=False)
        return (s["out"], *engine.cache_read(s["slot"], s["k_cache"], s["v_cache"], kv_scale=s["kv_scale"]))
    t.decode_planned_fp4(s["q"], s["k_cache"], s["v_cache"], s["kv_scale"], out=s["out"], want_lse=False)
    return (s["out"],)


def _run_write_plain(s):
    dtype, slot = s["case"]["dtype"], s["slot"].long()
    k = _rotate(s["k_new"], s["pos"][:, None], s["case"]["theta"]).transpose(1, 2)  # [layers, Hkv, n, D]
    v = s["v_new"].float().transpose(1, 2)
    if dtype == FP4:
        for i, x in enumerate((k, v)):
            code, scale = _encode(x)
            s["v_cache" if i else "k_cache"][:, :, slot] = _pack(code)
            s["kv_scale"][:, :, slot, i] = scale
        return _read_plain(s, s["k_cache"], s["v_cache"], s["kv_scale"])
    if dtype == FP8:
        k = (k / s["k_scale"][:, :, None, None]).clamp(-448, 448)
        v = (v / s["v_scale"][:, :, None, None]).clamp(-448, 448)
        s["k_cache"].view(torch.uint8)[:, :, slot] = k.to(TORCH[FP8]).view(torch.uint8)
        s["v_cache"].view(torch.uint8)[:, :, slot] = v.to(TORCH[FP8]).view(torch.uint8)
    else:
        s["k_cache"][:, :, slot] = k.to(TORCH[dtype])
        s["v_cache"][:, :, slot] = v.to(TORCH[dtype])
    return s["k_cache"], s["v_cache"]


def _run_write_own(s):
    from concurrent_shared_kv_gb300 import engine
    engine.cache_write(s["k_new"], s["v_new"], s["slot"], s["pos"], s["k_cache"], s["v_cache"],
                       rope_theta=s["case"]["theta"], k_scale=s.get("k_scale"), v_scale=s.get("v_scale"),
                       kv_scale=s.get("kv_scale"))
    if s["case"]["dtype"] == FP4:
        return _read_own(s, s["k_cache"], s["v_cache"], s["kv_scale"])
    return s["k_cache"], s["v_cache"]


def _run_commit_plain(s):
    src, dst = s["src"], s["dst"]
    k = _rotate(_values(s["k_src"][:, :, src], s["scale_src"][:, :, src, 0]), s["delta"], s["case"]["theta"])
    code, scale = _encode(k)
    s["k_dst"][:, :, dst] = _pack(code)
    s["scale_dst"][:, :, dst, 0] = scale
    s["v_dst"][:, :, dst] = s["v_src"][:, :, src]
    s["scale_dst"][:, :, dst, 1] = s["scale_src"][:, :, src, 1]
    return _read_plain(s, s["k_dst"], s["v_dst"], s["scale_dst"])


def _run_commit_own(s):
    from concurrent_shared_kv_gb300 import engine
    engine.block_commit_fp4(s["k_src"], s["v_src"], s["scale_src"], s["k_dst"], s["v_dst"], s["scale_dst"],
                            s["begin"], s["lens"], s["to"], s["to"], rope_theta=s["case"]["theta"])
    return _read_own(s, s["k_dst"], s["v_dst"], s["scale_dst"])


def _move_plain(pool, src, dst):
    bits = pool.view(torch.uint8)
    bits[:, :, dst] = bits[:, :, src]


def _run_move_plain(s):
    _move_plain(s["k_cache"], s["src"], s["dst"])
    _move_plain(s["v_cache"], s["src"], s["dst"])
    if s["case"]["dtype"] == FP4:
        _move_plain(s["kv_scale"], s["src"], s["dst"])
        return _read_plain(s, s["k_cache"], s["v_cache"], s["kv_scale"])
    return s["k_cache"], s["v_cache"]


def _run_move_own(s):
    from concurrent_shared_kv_gb300 import engine
    engine.block_move(s["k_cache"], s["v_cache"], s["begin"], s["lens"], s["to"], kv_scale=s.get("kv_scale"))
    if s["case"]["dtype"] == FP4:
        return _read_own(s, s["k_cache"], s["v_cache"], s["kv_scale"])
    return s["k_cache"], s["v_cache"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"decode": _run_decode_own, "write": _run_write_own, "commit": _run_commit_own,
                "move": _run_move_own}[op](state)
    return {"decode": _run_decode_plain, "write": _run_write_plain, "commit": _run_commit_plain,
            "move": _run_move_plain}[op](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    if case["op"] == "decode":
        P, W, T = case["problems"], case["workers"], case["chunk"]
        f = 0.625 if case["ragged"] else 1.0  # a ragged length's mean, of a quarter to the whole
        blocks = sum(max(1, T, case["block"] * (W - w) // W) for w in range(W)) * f
        tokens, rows = case["common"] * f + blocks, P * W * max(1, T)
        nbytes = P * tokens * case["hkv"] * 2 * ROW[FP4] + rows * 2 * case["hq"] * 256
        if case["append"]:
            nbytes += rows * case["hkv"] * 2 * (256 + ROW[FP4])
        return {"bytes": nbytes, "flops": 4 * 128 * case["hq"] * rows * tokens}
    if case["op"] == "write":
        rows = case["layers"] * case["rows"] * case["tokens"] * case["hkv"]
        act = case["d"] * (4 if case["dtype"] == F32 else 2)
        stored = ROW[case["dtype"]] * case["d"] // 128
        back = act + stored if case["dtype"] == FP4 else 0  # read back as values
        return {"bytes": 2 * rows * (act + stored + back), "flops": rows * case["d"] * 3}
    if case["op"] == "commit":
        tokens = case["tokens"] * (case["steps"] if case["steps"] == 1 else 0.75 * case["steps"])
        rows = case["layers"] * case["hkv"] * tokens
        return {"bytes": 2 * rows * (2 * ROW[FP4] + ROW[FP4] + 256), "flops": rows * 128 * 3}
    n = case["blocks"] * case["block"]
    # a fork reads its block once
    read, written, room = (case["block"], n, case["block"] + n) if case["kind"] == "fork" else (0.75 * n, 0.75 * n, 2 * n)
    row = ROW[case["dtype"]] * case["d"] // 128
    back = room * (row + 256) if case["dtype"] == FP4 else 0  # read back as values
    return {"bytes": 2 * case["layers"] * case["hkv"] * ((read + written) * row + back), "flops": 0}


# --------------------------------------------------------------------------
# the operators' definitions in 64 bits
# --------------------------------------------------------------------------

def _spin(x, pos, theta):
    """Complex rotation of x [..., D] (64 bits) by pos [...]."""
    half = x.shape[-1] // 2
    freq = torch.tensor([theta ** (-2.0 * i / (2 * half)) for i in range(half)], dtype=torch.float64, device=x.device)
    z = torch.complex(x[..., :half], x[..., half:])
    angle = pos.double()[..., None] * freq
    z = z * torch.polar(torch.ones_like(angle), angle)
    return torch.cat([z.real, z.imag], -1)


def _nearest(x):
    """x [..., D] in 64 bits as the 4-bit format holds it: the value of the
    nearest level under the vector's scale."""
    scale = (x.abs().amax(-1) / 6.0).float().to(torch.bfloat16).double()[..., None]
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    r = x.abs() / scale
    up = torch.searchsorted(level, r.contiguous()).clamp(1, 7)
    lo, hi = level[up - 1], level[up]
    to_hi = (r - lo > hi - r) | ((r - lo == hi - r) & (up % 2 == 0))
    return torch.where(to_hi, hi, lo) * x.sign() * scale


def _values64(codes, scale):
    sign = 1.0 - 2.0 * torch.stack([codes & 8, codes >> 4 & 8], -1).bool().double()
    e = torch.stack([codes >> 1 & 3, codes >> 5 & 3], -1).double()
    m = torch.stack([codes & 1, codes >> 4 & 1], -1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * 2 ** (e - 1))
    return (sign * mag).flatten(-2) * scale.double()[..., None]


def _exact_decode(case, seed):
    s = _prepare_decode(case, seed)
    L, hq, hkv, theta = s["layout"], case["hq"], case["hkv"], case["theta"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    k64, v64 = _values64(s["k_cache"], s["kv_scale"][..., 0]), _values64(s["v_cache"], s["kv_scale"][..., 1])
    new = []
    if case["append"]:
        kn = _nearest(_spin(s["k_new"].double(), s["at"][:, None], theta))
        vn = _nearest(s["v_new"].double())
        k64[:, s["slot"].long()], v64[:, s["slot"].long()] = kn.transpose(0, 1), vn.transpose(0, 1)
        new = [kn, vn]
    for r, view in enumerate(L["views"]):
        q = s["q"][r].double()
        parts, values = [], []
        for b, off, lim in zip(view, L["offs"][r], L["limits"][r]):  # the query turned to each block's positions
            n = L["lens"][b] if lim < 0 else min(lim, L["lens"][b])
            qb = _spin(q, torch.tensor(L["q_pos"][r] - off, device="cuda"), theta).reshape(hkv, hq // hkv, 128)
            at = L["starts"][b]
            parts.append(torch.einsum("hgd,hld->hgl", qb, k64[:, at:at + n]))
            values.append(v64[:, at:at + n])
        weight = torch.softmax(torch.cat(parts, -1) * 128 ** -0.5, -1)
        out[r] = torch.einsum("hgl,hld->hgd", weight, torch.cat(values, 1)).reshape(hq, 128)
    return (out, *new)


def _exact_write(case, seed):
    s = _prepare_write(case, seed)
    k = _spin(s["k_new"].double(), s["pos"][:, None], case["theta"])
    v = s["v_new"].double()
    if case["dtype"] == FP4:
        return _nearest(k), _nearest(v)
    kd = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device="cuda")
    vd = torch.zeros_like(kd)
    if case["dtype"] == FP8:  # in units of the heads' scales
        k, v = k / s["k_scale"].double()[:, None, :, None], v / s["v_scale"].double()[:, None, :, None]
        k, v = k.clamp(-448, 448).float().to(TORCH[FP8]).double(), v.clamp(-448, 448).float().to(TORCH[FP8]).double()
    kd[:, :, s["slot"].long()], vd[:, :, s["slot"].long()] = k.transpose(1, 2), v.transpose(1, 2)
    return kd, vd


def _exact_commit(case, seed):
    s = _prepare_commit(case, seed)
    k_out = torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda")
    v_out, at = torch.zeros_like(k_out), s["dst"] - case["history"]
    for l in range(case["layers"]):
        k = _values64(s["k_src"][l][:, s["src"]], s["scale_src"][l][:, s["src"], 0])
        k_out[l, at] = _nearest(_spin(k, s["delta"], case["theta"])).transpose(0, 1)
        v_out[l, at] = _values64(s["v_src"][l][:, s["src"]], s["scale_src"][l][:, s["src"], 1]).transpose(0, 1)
    return k_out, v_out


def _exact_move(case, seed):
    s = _prepare_move(case, seed)
    for c in (s["k_cache"], s["v_cache"], s.get("kv_scale")):
        for b, m, to in zip(s["begin"], s["lens"], s["to"]):  # one move after the other
            if c is not None:
                c[:, :, to:to + m] = c[:, :, b:b + m].clone()
    if case["dtype"] != FP4:
        return s["k_cache"], s["v_cache"]
    return [_values64(c, s["kv_scale"][..., i]).transpose(1, 2) for i, c in enumerate((s["k_cache"], s["v_cache"]))]


def exact(case, seed):
    return {"decode": _exact_decode, "write": _exact_write, "commit": _exact_commit,
            "move": _exact_move}[case["op"]](case, seed)
