"""Measured cases of the draft-tree operators: attention for a tree of drafted
tokens over the shared cache, verification of the drafted tokens against the
target's probabilities, and the commit of the accepted path.

With ``own`` false the operators run in their plain form (elementary torch
operations, 32 bits or more whatever the storage type); with ``own`` true they
run through the library's entry points.
"""
import math

import torch

own = False

F32, BF16, FP8 = "f32", "bf16", "fp8"
TORCH = {F32: torch.float32, BF16: torch.bfloat16, FP8: torch.float8_e4m3fn}
BYTES = {F32: 4, BF16: 2, FP8: 1}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _tree(name, dtype, problems, workers, hq, hkv, d, common, block, nodes, branch, ragged=False, theta=1e6):
    return {"name": name, "op": "tree", "dtype": dtype, "problems": problems, "workers": workers, "hq": hq,
            "hkv": hkv, "d": d, "common": common, "block": block, "nodes": nodes, "branch": branch,
            "ragged": ragged, "theta": theta}


def _verify(name, dtype, rows, nodes, vocab, branch, drafted):
    return {"name": name, "op": "verify", "dtype": dtype, "rows": rows, "nodes": nodes, "vocab": vocab,
            "branch": branch, "drafted": drafted}


def _commit(name, dtype, layers, rows, hkv, d, nodes, block):
    return {"name": name, "op": "commit", "dtype": dtype, "layers": layers, "rows": rows, "hkv": hkv, "d": d,
            "nodes": nodes, "block": block}


def listed():
    return [
        # two workers at the start of a small fp32 model's answer: latency
        _tree("tree-tiny-f32", F32, 1, 2, 4, 2, 64, 256, 40, 6, 2, theta=1e4),
        # a short prompt, a chain of four drafted tokens (no branches): latency
        _tree("tree-chain-short", BF16, 1, 2, 40, 8, 128, 1001, 250, 4, 1),
        # four workers on a 16K history, a small tree: the ordinary step
        _tree("tree-16-history-16k", BF16, 1, 4, 40, 8, 128, 16384, 512, 16, 3),
        # the same with a large tree: arithmetic counts as much as memory
        _tree("tree-64-history-16k", BF16, 1, 4, 40, 8, 128, 16384, 512, 64, 4),
        # four workers on a 32K history in 8-bit codes
        _tree("tree-24-history-32k-fp8", FP8, 1, 4, 32, 8, 128, 32768, 1024, 24, 2),
        # a batch of independent problems of unlike lengths and unlike trees
        _tree("tree-serve-ragged", BF16, 8, 4, 40, 8, 128, 32768, 1024, 8, 2, ragged=True),
        # one group of workers, drafts sampled from the draft model
        _verify("verify-group", F32, 4, 16, 131072, 3, "sampled"),
        # a large batch in 16 bits
        _verify("verify-batch-bf16", BF16, 64, 8, 131072, 2, "sampled"),
        # a small odd vocabulary, a wide tree of the draft model's top choices
        _verify("verify-top-choices", F32, 4, 64, 50021, 4, "chosen"),
        # accepted tokens of four workers moved in all layers of a large model
        _commit("commit-group", BF16, 64, 4, 8, 128, 16, 512),
        # the same of a large batch over 8-bit caches
        _commit("commit-batch-fp8", FP8, 36, 64, 8, 128, 24, 200),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "verify", "verify", "commit"])
    if op == "tree":
        dtype = rng.choice([F32, BF16, BF16, BF16, FP8])
        heads = rng.choice([(40, 8), (32, 8), (4, 2), (8, 8), (16, 1)])
        d = rng.choice([64, 128]) if dtype == F32 else 128 if dtype == FP8 else rng.choice([64, 128, 128])
        slow = dtype == F32 or d == 64
        problems = rng.choice([1, 1, 2, 3]) if slow else rng.choice([1, 1, 1, 2, 5, 8])
        workers = rng.choice([1, 2, 3, 4] if problems > 3 else [1, 2, 3, 4, 6])
        nodes = _spread(rng, 1, 16 if slow or problems > 3 else 100)
        common = _spread(rng, 64, 4096 if slow else 32768 if problems > 1 or nodes > 64 else 65536)
        block = _spread(rng, 1, 1024)
        nodes = max(1, min(nodes, int(1.8e8 / (problems * workers * heads[0] * (common + workers * block)))))
        c = _tree("", dtype, problems, workers, heads[0], heads[1], d, common, block, nodes,
                  rng.choice([1, 2, 3, 5]), rng.random() < 0.5, rng.choice([1e4, 1e6]))
    elif op == "verify":
        rows = _spread(rng, 1, 64)
        c = _verify("", rng.choice([F32, BF16]), rows, _spread(rng, 1, min(64, 512 // rows)), _spread(rng, 1000, 131072),
                    rng.choice([1, 2, 4]), rng.choice(["sampled", "chosen"]))
    else:
        c = _commit("", rng.choice([F32, BF16, FP8]), _spread(rng, 1, 48), _spread(rng, 1, 32), rng.choice([1, 2, 8]),
                    rng.choice([64, 128]), _spread(rng, 1, 64), _spread(rng, 1, 300))
        if c["dtype"] == FP8:
            c["d"] = 128
    del c["name"]
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _trees(g, rows, nodes, branch, ragged):
    """Node counts and parents: node 0 is the root; about `branch` children a
    node, level by level (branch 1: a chain).  Host lists."""
    n_nodes, parent = [], []
    for r in range(rows):
        n = nodes
        if ragged:
            n = int(torch.randint(max(1, nodes // 3), nodes + 1, (1,), generator=g))
        jump = torch.randint(0, branch + 1, (nodes,), generator=g).tolist()
        p = [-1]
        for i in range(1, n):
            p.append(min(i - 1, (i - 1) // branch + (jump[i] if branch > 1 else 0)))
        n_nodes.append(n)
        parent.append(p + [-1] * (nodes - n))
    return n_nodes, parent


def _int(x, dev="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _tree_layout(case, g):
    """Host lists: block lengths and starts, views, positions, trees, capacity."""
    P, W, T = case["problems"], case["workers"], case["nodes"]
    lens, starts, at = [], [], 0
    for p in range(P):
        c = case["common"]
        if case["ragged"]:
            c = int(torch.randint(max(1, c // 4), c + 1, (1,), generator=g))
        row = [c]
        for w in range(W):
            b = max(1, case["block"] * (W - w) // W)
            if case["ragged"]:
                b = int(torch.randint(max(1, b // 4), b + 1, (1,), generator=g))
            row.append(b)
        for n in row:
            lens.append(n)
            starts.append(at)
            at += n
    views, offs, q_pos, tree_block = [], [], [], []
    for p in range(P):
        base = p * (W + 1)
        for w in range(W):
            order = [base] + [base + 1 + o for o in range(W) if o != w] + [base + 1 + w]
            o, off = 0, []
            for b in order:
                off.append(o)
                o += lens[b]
            views.append(order)
            offs.append(off)
            q_pos.append(o)
            tree_block.append(base + 1 + w)
    n_nodes, parent = _trees(g, P * W, T, case["branch"], case["ragged"])
    tree_start = [at + r * T for r in range(P * W)]  # drafts: an area of their own behind the blocks
    # the pool itself has room for the longest blocks
    at = P * (case["common"] + sum(max(1, case["block"] * (W - w) // W) for w in range(W)))
    return dict(lens=lens, starts=starts, views=views, offs=offs, q_pos=q_pos, tree_block=tree_block,
                n_nodes=n_nodes, parent=parent, tree_start=tree_start, capacity=at + P * W * T)


def _prepare_tree(case, seed):
    g = torch.Generator().manual_seed(seed)
    L = _tree_layout(case, g)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    R, T, hq, hkv, d = case["problems"] * case["workers"], case["nodes"], case["hq"], case["hkv"], case["d"]
    act = torch.float32 if case["dtype"] == F32 else torch.bfloat16

    def normal(*shape):
        return torch.randn(shape, generator=gd, device="cuda", dtype=torch.float32)

    k, v = normal(hkv, L["capacity"], d), normal(hkv, L["capacity"], d)
    for p in range(case["problems"]):  # the first key of a history draws attention
        k[:, L["starts"][p * (case["workers"] + 1)]] *= 8.0
    s = {"case": case, "layout": L}
    if case["dtype"] == FP8:
        s["k_scale"] = k.abs().amax(dim=(1, 2)) / 448.0
        s["v_scale"] = v.abs().amax(dim=(1, 2)) / 448.0
        k, v = k / s["k_scale"][:, None, None], v / s["v_scale"][:, None, None]
    s["k_cache"], s["v_cache"] = k.to(TORCH[case["dtype"]]), v.to(TORCH[case["dtype"]])
    s["q"] = normal(R, T, hq, d).to(act)
    s["k_new"], s["v_new"] = normal(R, T, hkv, d).to(act), normal(R, T, hkv, d).to(act)
    s["out"] = torch.zeros(R, T, hq, d, dtype=act, device="cuda")
    # what the plain form indexes with: per row, the view's tokens (padded), their entries, ancestors, depths
    longest = max(sum(L["lens"][b] for b in view) for view in L["views"])
    n_view = len(L["views"][0])
    lens = _int([[L["lens"][b] for b in view] for view in L["views"]]).long()
    starts = _int([[L["starts"][b] for b in view] for view in L["views"]]).long()
    at = torch.arange(longest, device="cuda").expand(R, longest)
    ends = lens.cumsum(1)
    ent = torch.searchsorted(ends, at.contiguous(), right=True).clamp(max=n_view - 1)
    s["seen"] = at < ends[:, -1:]
    s["entry"] = ent
    s["token"] = torch.where(s["seen"], starts.gather(1, ent) + at - (ends - lens).gather(1, ent), 0)
    anc = torch.zeros(R, T, T, dtype=torch.bool)
    depth = torch.zeros(R, T, dtype=torch.int64)
    for r in range(R):
        for i in range(L["n_nodes"][r]):
            p = L["parent"][r][i]
            if p >= 0:
                anc[r, i] = anc[r, p]
                depth[r, i] = depth[r, p] + 1
            anc[r, i, i] = True
    s["ancestors"], s["depth"] = anc.cuda(), depth.cuda()
    s["offset"], s["position"] = _int(L["offs"]).long(), _int(L["q_pos"]).long()
    s["own_len"] = _int([L["lens"][b] for b in L["tree_block"]]).long()
    live = torch.arange(T)[None] < torch.tensor(L["n_nodes"])[:, None]
    s["live"] = live.cuda()
    s["live_at"] = live.reshape(-1).nonzero()[:, 0].cuda()
    s["slot"] = (torch.tensor(L["tree_start"])[:, None] + torch.arange(T))[live].cuda()
    if own:
        from concurrent_shared_kv_gb300 import engine
        t = engine.TreeSession(n_rows=R, max_nodes=T, n_q_heads=hq, n_kv_heads=hkv, head_dim=d,
                               n_blocks=len(L["lens"]), max_view_blocks=n_view, capacity=L["capacity"], dtype=act,
                               rope_theta=case["theta"], kv_fp8=case["dtype"] == FP8)
        t.set_metadata(L["starts"], L["lens"], L["views"], L["offs"], L["q_pos"])
        t.plan(L["tree_block"], L["n_nodes"], L["parent"], tree_start=L["tree_start"])
        s["session"] = t
    return s


def _verify_inputs(case, seed):
    """Target and draft distributions after every node (alike, as a good
    draft's are), trees, drafted tokens, and the random numbers."""
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    R, T, V = case["rows"], case["nodes"], case["vocab"]
    n_nodes, parent = _trees(g, R, T, case["branch"], True)
    logits = 3.0 * torch.randn(R, T, V, generator=gd, device="cuda")
    dt = TORCH[case["dtype"]]
    p = torch.softmax(logits, -1).to(dt)
    logits += 0.7 * torch.randn(R, T, V, generator=gd, device="cuda")
    q = torch.softmax(logits, -1).to(dt)
    at = torch.tensor(parent).clamp(min=0).cuda()
    if case["drafted"] == "sampled":  # children of a node are drawn from its draft distribution
        cum = q.double().cumsum(-1).reshape(R * T, V)
        u = torch.rand(R, T, generator=gd, device="cuda", dtype=torch.float64)
        rows = (torch.arange(R, device="cuda")[:, None] * T + at).reshape(-1)
        token = torch.stack([torch.searchsorted(cum[rows[i]], u.reshape(-1)[i] * cum[rows[i], -1], right=True)
                             for i in range(R * T)]).reshape(R, T).clamp(max=V - 1)
    else:  # the children of a node are its draft distribution's top choices, best first
        rank, seen = [], {}
        for r in range(R):
            for i in range(T):
                key = (r, parent[r][i])
                rank.append(seen.get(key, 0))
                seen[key] = rank[-1] + 1
        top = q.float().topk(min(V, max(rank) + 1), -1).indices
        rank = torch.tensor(rank).reshape(R, T).cuda().clamp(max=top.shape[-1] - 1)
        token = top[torch.arange(R, device="cuda")[:, None], at, rank]
    s = {"p": p, "q": q if case["drafted"] == "sampled" else None, "token": token.int(),
         "n_nodes": _int(n_nodes), "parent": _int(parent),
         "u_accept": torch.rand(R, T, generator=gd, device="cuda"), "u_sample": torch.rand(R, generator=gd, device="cuda")}
    return s


def _prepare_verify(case, seed):
    s = _verify_inputs(case, seed)
    R, T = case["rows"], case["nodes"]
    s["case"] = case
    s["path"] = torch.empty(R, T, dtype=torch.int32, device="cuda")
    s["n_path"] = torch.empty(R, dtype=torch.int32, device="cuda")
    s["next_token"] = torch.empty(R, dtype=torch.int32, device="cuda")
    return s


def _prepare_commit(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    R, T, hkv, d, layers = case["rows"], case["nodes"], case["hkv"], case["d"], case["layers"]
    # each row: a block with room for its accepted tokens, then the drafts' own area
    lens = torch.randint(max(1, case["block"] // 4), case["block"] + 1, (R,), generator=g).tolist()
    starts, at = [], 0
    for n in lens:
        starts.append(at)
        at += n + T
    tree_start = [at + r * T for r in range(R)]
    capacity = R * (case["block"] + 2 * T)  # room for the longest blocks
    n_nodes, parent = _trees(g, R, T, 3, False)
    n_path, path = [], []
    for r in range(R):  # the path from the root to a random node
        i = int(torch.randint(0, n_nodes[r], (1,), generator=g))
        line = []
        while i >= 0:
            line.append(i)
            i = parent[r][i]
        line = line[::-1][:8]
        n_path.append(len(line))
        path.append(line + [-1] * (T - len(line)))
    s = {"case": case, "path": _int(path), "n_path": _int(n_path)}
    shape = (layers, hkv, capacity, d)
    dt = TORCH[case["dtype"]]
    s["k_cache"] = torch.empty(shape, dtype=dt, device="cuda")
    s["v_cache"] = torch.empty(shape, dtype=dt, device="cuda")
    for l in range(layers):
        for c in (s["k_cache"], s["v_cache"]):
            c[l] = torch.randn(shape[1:], generator=gd, device="cuda").to(dt)
    s["end"] = (_int(starts) + _int(lens)).long()
    s["tree_start"] = _int(tree_start).long()
    if own:
        from concurrent_shared_kv_gb300 import engine
        t = engine.TreeSession(n_rows=R, max_nodes=T, n_q_heads=hkv, n_kv_heads=hkv, head_dim=d, n_blocks=R,
                               max_view_blocks=1, capacity=capacity,
                               dtype=torch.float32 if case["dtype"] == F32 else torch.bfloat16, rope_theta=1e6,
                               kv_fp8=case["dtype"] == FP8)
        t.set_metadata(starts, lens, [[r] for r in range(R)], [[0] for r in range(R)], lens)
        t.plan(list(range(R)), n_nodes, parent, tree_start=tree_start)
        s["session"] = t
    return s


def prepare(case, seed):
    return {"tree": _prepare_tree, "verify": _prepare_verify, "commit": _prepare_commit}[case["op"]](case, seed)


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


def _run_tree_plain(s):
    case, theta = s["case"], s["case"]["theta"]
    R, T, hq, hkv, d = case["problems"] * case["workers"], case["nodes"], case["hq"], case["hkv"], case["d"]
    k_cache, v_cache = s["k_cache"], s["v_cache"]
    # the new tokens into the cache: keys rotated at their positions in their block
    k_new = _rotate(s["k_new"], (s["own_len"][:, None] + s["depth"])[..., None], theta)
    v_new = s["v_new"].float()
    if case["dtype"] == FP8:
        k_new = (k_new / s["k_scale"][:, None]).clamp(-448, 448)
        v_new = (v_new / s["v_scale"][:, None]).clamp(-448, 448)
    k_new, v_new = k_new.to(k_cache.dtype), v_new.to(v_cache.dtype)
    k_cache[:, s["slot"]] = k_new.reshape(R * T, hkv, d)[s["live_at"]].transpose(0, 1)
    v_cache[:, s["slot"]] = v_new.reshape(R * T, hkv, d)[s["live_at"]].transpose(0, 1)
    # every row's keys at their positions in its view, [R, Hkv, L + T, D]
    k = k_cache[:, s["token"]].transpose(0, 1).float()
    v = v_cache[:, s["token"]].transpose(0, 1).float()
    k = _rotate(k, s["offset"].gather(1, s["entry"])[:, None], theta)
    k_tree = _rotate(k_new.transpose(1, 2), (s["position"] - s["own_len"])[:, None, None], theta)
    k = torch.cat([k, k_tree], 2)
    v = torch.cat([v, v_new.transpose(1, 2).float()], 2)
    if case["dtype"] == FP8:
        k, v = k * s["k_scale"][:, None, None], v * s["v_scale"][:, None, None]
    q = _rotate(s["q"], (s["position"][:, None] + s["depth"])[..., None], theta)
    q = q.reshape(R, T, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4)  # [R, Hkv, T, G, D]
    score = q.reshape(R, hkv, -1, d) @ k.transpose(2, 3) * d ** -0.5
    score = score.reshape(R, hkv, T, hq // hkv, -1)
    mask = torch.cat([s["seen"][:, None].expand(-1, T, -1), s["ancestors"]], 2)
    score = score.masked_fill(~mask[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    e = (score - top).exp()
    total = e.sum(-1, keepdim=True)
    out = (e.reshape(R, hkv, -1, e.shape[-1]) @ v).reshape(R, hkv, T, hq // hkv, d) / total
    out = out.permute(0, 2, 1, 3, 4).reshape(R, T, hq, d)
    s["out"].copy_(torch.where(s["live"][..., None, None], out, 0))
    return s["out"], k_cache, v_cache


def _run_tree_own(s):
    t = s["session"]
    if s["case"]["dtype"] == FP8:
        t.decode_fp8(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                     out=s["out"], want_lse=False)
    else:
        t.decode(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], out=s["out"], want_lse=False)
    return s["out"], s["k_cache"], s["v_cache"]


def _run_verify_plain(s):
    p, q, token, parent = s["p"], s["q"], s["token"].long(), s["parent"].long()
    R, T, V = p.shape
    rows = torch.arange(R, device=p.device)
    cur = torch.zeros(R, dtype=torch.int64, device=p.device)
    on_path = torch.zeros(R, T, dtype=torch.bool, device=p.device)
    on_path[:, 0] = s["n_nodes"] > 0
    c = torch.zeros(R, dtype=torch.float64, device=p.device)
    mass = torch.ones_like(c)
    gone = torch.zeros(R, V, dtype=torch.bool, device=p.device)
    # nodes in index order: a node's children come after it, and each test depends on the ones before it
    for i in range(1, T):
        here = (parent[:, i] == cur) & (i < s["n_nodes"])
        x = token[:, i]
        px = p[rows, cur, x].double()
        if q is None:
            a = torch.where(gone[rows, x], 0.0, px)
            ok = here & (s["u_accept"][:, i].double() * mass < a)
            no = here & ~ok
            mass = torch.where(no, (mass - a).clamp(min=0), mass)
            gone[rows, x] |= no
        else:
            qx = q[rows, cur, x].double()
            a = (px - c * qx).clamp(min=0)
            ok = here & (s["u_accept"][:, i].double() * qx * mass < a)
            left = (p[rows, cur].double() - (c + mass)[:, None] * q[rows, cur].double()).clamp(min=0).sum(-1)
            no = here & ~ok & (left > 0)
            c, mass = torch.where(no, c + mass, c), torch.where(no, left, mass)
        cur = torch.where(ok, i, cur)
        on_path[:, i] = ok
        c, mass = torch.where(ok, 0.0, c), torch.where(ok, 1.0, mass)
        gone &= ~ok[:, None]
    a = p[rows, cur].double()
    a = torch.where(gone, 0.0, a) if q is None else (a - c[:, None] * q[rows, cur].double()).clamp(min=0)
    cum = a.cumsum(-1)
    total = cum[:, -1]
    next_token = (cum <= (s["u_sample"].double() * total)[:, None]).sum(-1).clamp(max=V - 1)
    next_token = torch.where((total > 0) & (s["n_nodes"] > 0), next_token, -1)
    order = torch.where(on_path, torch.arange(T, device=p.device), T).sort(-1).values
    s["path"].copy_(torch.where(order < T, order, -1))
    s["n_path"].copy_(on_path.sum(-1))
    s["next_token"].copy_(next_token)
    return s["path"], s["n_path"], s["next_token"]


def _run_verify_own(s):
    from concurrent_shared_kv_gb300 import engine
    return engine.tree_verify(s["n_nodes"], s["parent"], s["token"], s["p"], s["q"], s["u_accept"], s["u_sample"],
                              path=s["path"], n_path=s["n_path"], next_token=s["next_token"])


def _run_commit_plain(s):
    T = s["case"]["nodes"]
    j = torch.arange(T, device="cuda")
    keep = j[None] < s["n_path"][:, None]
    # slots past the path copy onto themselves
    src = torch.where(keep, s["tree_start"][:, None] + s["path"], s["tree_start"][:, None] + j).reshape(-1)
    dst = torch.where(keep, s["end"][:, None] + j, s["tree_start"][:, None] + j).reshape(-1)
    for cache in (s["k_cache"], s["v_cache"]):
        bits = cache.view(torch.uint8)
        bits[:, :, dst] = bits[:, :, src]
    return s["k_cache"], s["v_cache"]


def _run_commit_own(s):
    s["session"].commit(s["k_cache"], s["v_cache"], s["path"], s["n_path"])
    return s["k_cache"], s["v_cache"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _run_tree_own, "verify": _run_verify_own, "commit": _run_commit_own}[op](state)
    return {"tree": _run_tree_plain, "verify": _run_verify_plain, "commit": _run_commit_plain}[op](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    if case["op"] == "tree":
        P, W, T = case["problems"], case["workers"], case["nodes"]
        # the expected lengths of a ragged case: three quarters of a node range from a third, five eighths of a length
        f, fn = (0.625, 2 / 3) if case["ragged"] else (1.0, 1.0)
        blocks = sum(max(1, case["block"] * (W - w) // W) for w in range(W)) * f
        tokens = P * (case["common"] * f + blocks)
        rows = P * W * T * fn
        esz, act = BYTES[case["dtype"]], 4 if case["dtype"] == F32 else 2
        kv = 2 * case["hkv"] * case["d"]
        nbytes = tokens * kv * esz + rows * (2 * case["hq"] * case["d"] * act + kv * (act + esz))
        flops = 4 * case["d"] * case["hq"] * rows * (case["common"] * f + blocks + T * fn / 2)
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "verify":
        # the last node's rows: the target's, and the draft's where tokens were sampled from it
        each = case["vocab"] * BYTES[case["dtype"]] * (2 if case["drafted"] == "sampled" else 1)
        return {"bytes": case["rows"] * (each + case["nodes"] * 16), "flops": case["rows"] * case["vocab"] * 3}
    accepted = min(8, 1 + case["nodes"] / 4)
    row = case["layers"] * case["hkv"] * case["d"] * BYTES[case["dtype"]]
    return {"bytes": case["rows"] * accepted * row * 4, "flops": 0}


# --------------------------------------------------------------------------
# the operators' definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_tree(case, seed):
    s = _prepare_tree(case, seed)
    L, d, hq, hkv = s["layout"], case["d"], case["hq"], case["hkv"]
    G, half, dev = hq // hkv, d // 2, "cuda"
    freq = torch.tensor([case["theta"] ** (-2.0 * i / d) for i in range(half)], dtype=torch.float64, device=dev)

    def spin(x, pos):  # complex rotation of x [N, H, D] by pos [N]
        z = torch.complex(x[..., :half].double(), x[..., half:].double())
        z = z * torch.polar(torch.ones_like(freq), pos.double()[:, None] * freq)[:, None]
        return torch.cat([z.real, z.imag], -1)

    fp8 = case["dtype"] == FP8
    ks = s["k_scale"].double() if fp8 else torch.ones(hkv, dtype=torch.float64, device=dev)
    vs = s["v_scale"].double() if fp8 else torch.ones(hkv, dtype=torch.float64, device=dev)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=dev)
    k64, v64 = s["k_cache"].double(), s["v_cache"].double()
    for r, view in enumerate(L["views"]):
        n = L["n_nodes"][r]
        depth = s["depth"][r, :n]
        base = L["lens"][L["tree_block"][r]]
        kn = spin(s["k_new"][r, :n], base + depth)
        vn = s["v_new"][r, :n].double()
        at = L["tree_start"][r]
        if fp8:  # the attended values are the stored ones
            kn = (kn / ks[:, None]).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
            vn = (vn / vs[:, None]).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
        elif case["dtype"] == BF16:
            kn = kn.float().to(torch.bfloat16).double()
        k64[:, at:at + n], v64[:, at:at + n] = kn.transpose(0, 1), vn.transpose(0, 1)
        q = s["q"][r, :n]
        parts, values = [], []
        for b, off in zip(view, L["offs"][r]):  # the query turned to each block's positions
            qb = spin(q, L["q_pos"][r] - off + depth).reshape(n, hkv, G, d)
            lo, hi = L["starts"][b], L["starts"][b] + L["lens"][b]
            parts.append(torch.einsum("nhgd,hld->nhgl", qb, k64[:, lo:hi] * ks[:, None, None]))
            values.append(v64[:, lo:hi])
        qt = spin(q, base + depth).reshape(n, hkv, G, d)
        tree = torch.einsum("nhgd,hld->nhgl", qt, k64[:, at:at + n] * ks[:, None, None])
        parts.append(tree.masked_fill(~s["ancestors"][r, :n, :n][:, None, None], -math.inf))
        values.append(v64[:, at:at + n])
        weight = torch.softmax(torch.cat(parts, -1) * d ** -0.5, -1)
        o = torch.einsum("nhgl,hld->nhgd", weight, torch.cat(values, 1) * vs[:, None, None])
        out[r, :n] = o.reshape(n, hq, d)
    return out, k64, v64


def _exact_verify(case, seed):
    s = _verify_inputs(case, seed)
    R, T, V = s["p"].shape
    paths, counts, tokens = [], [], []
    for r in range(R):
        n, parent, token = int(s["n_nodes"][r]), s["parent"][r].tolist(), s["token"][r].tolist()
        u = s["u_accept"][r].double().tolist()
        at, line = 0, [0]
        while True:  # at each node the residual distribution, normalised anew after each rejection
            dist = s["p"][r, at].double()
            took = None
            for i in [i for i in range(at + 1, n) if parent[i] == at]:
                x = token[i]
                if s["q"] is None:
                    if u[i] < float(dist[x]):
                        took = i
                        break
                    rest = 1.0 - float(dist[x])
                    dist = dist.clone()
                    dist[x] = 0.0
                    dist = dist / rest if rest > 0 else dist
                else:
                    draft = s["q"][r, at].double()
                    if u[i] * float(draft[x]) < float(dist[x]):
                        took = i
                        break
                    rest = (dist - draft).clamp(min=0)
                    if float(rest.sum()) > 0:
                        dist = rest / rest.sum()
            if took is None:
                break
            at = took
            line.append(at)
        cum = dist.cumsum(0)
        x = int((cum <= float(s["u_sample"][r]) * cum[-1]).sum())
        paths.append(line + [-1] * (T - len(line)))
        counts.append(len(line))
        tokens.append(min(x, V - 1))
    return _int(paths), _int(counts), _int(tokens)


def _exact_commit(case, seed):
    s = _prepare_commit(case, seed)
    for cache in (s["k_cache"], s["v_cache"]):
        for r, n in enumerate(s["n_path"].tolist()):  # token after token, from the drafts' area to the block's end
            for j in range(n):
                at = int(s["tree_start"][r]) + int(s["path"][r, j])
                cache[:, :, int(s["end"][r]) + j] = cache[:, :, at].clone()
    return s["k_cache"], s["v_cache"]


def exact(case, seed):
    if case["op"] == "tree":
        return _exact_tree(case, seed)
    if case["op"] == "verify":
        return _exact_verify(case, seed)
    return _exact_commit(case, seed)
