"""GPU tests of the draft-tree operators against their definitions in float64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from concurrent_shared_kv_gb300 import api, engine
from tests import tree_ref as ref

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}
# half a step of each type, relative to the value
STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp8": 2.0 ** -4}


class Tree:
    """One seeded step: pools on the device, metadata, trees, new tokens."""

    def __init__(self, dtype="bf16", hq=10, hkv=2, d=128, lens=(300, 40, 129), views=None, T=5, n_nodes=None,
                 kind="tree", tree_block=None, in_place=False, seed=0, theta=1e4, scale=None, shuffle=False,
                 poison=True, parent=None):
        rng = np.random.Generator(np.random.PCG64(seed))
        self.dtype, self.hq, self.hkv, self.d, self.T, self.theta = dtype, hq, hkv, d, T, theta
        self.scale = d ** -0.5 if scale is None else scale
        W = len(lens) - 1
        self.block_len = np.asarray(lens, np.int32)
        if views is None:  # the combined layout of one problem
            views = api.views_combined(self.block_len, 1, W)
        self.view_block, self.view_offset, self.q_pos = [np.asarray(x, np.int32) for x in views]
        R = self.R = self.view_block.shape[0]
        self.tree_block = np.arange(1, R + 1, dtype=np.int32) if tree_block is None else np.asarray(tree_block, np.int32)
        self.n_nodes = np.full(R, T, np.int32) if n_nodes is None else np.asarray(n_nodes, np.int32)
        self.parent = ref.random_parents(rng, R, T, kind, self.n_nodes) if parent is None else np.asarray(parent, np.int32)
        # blocks with gaps of T + 3 slots, then the trees' own area, back to front
        gap = T + 3
        self.block_start = (np.cumsum(self.block_len + gap) - self.block_len).astype(np.int32)
        end = int((self.block_len + gap).sum()) + gap
        self.in_place = in_place
        if in_place:
            self.tree_start = (self.block_start + self.block_len)[self.tree_block]
        else:
            self.tree_start = (end + (R - 1 - np.arange(R)) * (T + 1)).astype(np.int32)
        self.cap = end + R * (T + 1) + 5
        self.heads = np.repeat(np.arange(hkv), hq // hkv).astype(np.int32)
        if shuffle:
            rng.shuffle(self.heads)
        self.shuffle = shuffle
        # values outside every block are poison
        k = np.full((hkv, self.cap, d), np.nan if poison else 0.0)
        v = k.copy()
        for s, n in zip(self.block_start, self.block_len):
            k[:, s:s + n] = rng.standard_normal((hkv, n, d))
            v[:, s:s + n] = rng.standard_normal((hkv, n, d))
        tdt = TORCH[dtype]
        self.k_scale = self.v_scale = None
        if dtype == "fp8":
            # scales that are no powers of two; the largest key lands at 448
            ks = np.nanmax(np.abs(k), axis=(1, 2), initial=1.0) / 448
            vs = np.nanmax(np.abs(v), axis=(1, 2), initial=1.0) / 448
            self.k_scale, self.v_scale = ref.dev(ks, torch.float32), ref.dev(vs, torch.float32)
            self.k = ref.dev(k, torch.float32).div(self.k_scale[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.v = ref.dev(v, torch.float32).div(self.v_scale[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            self.k, self.v = ref.dev(k, tdt), ref.dev(v, tdt)

        def new(h):  # entries behind a row's nodes are poison too
            x = rng.standard_normal((R, T, h, d))
            for r in range(R):
                x[r, max(0, int(self.n_nodes[r])):] = np.nan
            return ref.dev(x, tdt)
        self.q, self.k_new, self.v_new = new(hq), new(hkv), new(hkv)

    def session(self):
        s = engine.TreeSession(n_rows=self.R, max_nodes=self.T, n_q_heads=self.hq, n_kv_heads=self.hkv,
                               head_dim=self.d, n_blocks=len(self.block_len),
                               max_view_blocks=self.view_block.shape[1], capacity=self.cap, dtype=TORCH[self.dtype],
                               rope_theta=self.theta, scale=self.scale, kv_fp8=self.dtype == "fp8")
        s.set_metadata(self.block_start, self.block_len, self.view_block, self.view_offset, self.q_pos,
                       self.heads if self.shuffle else None)
        self.plan(s)
        return s

    def plan(self, s):
        s.plan(self.tree_block, self.n_nodes, self.parent, tree_start=None if self.in_place else self.tree_start)

    def run(self, s, out=None, lse=None):
        if self.dtype == "fp8":
            return s.decode_fp8(self.q, self.k_new, self.v_new, self.k, self.v, self.k_scale, self.v_scale, out=out, lse=lse)
        return s.decode(self.q, self.k_new, self.v_new, self.k, self.v, out=out, lse=lse)

    def stored(self, x, scale):
        x = ref.to_np(x.float()) if self.dtype == "fp8" else ref.to_np(x)
        return x * (1.0 if scale is None else ref.to_np(scale)[:, None, None])

    def expected_tokens(self, rows):
        """Exact values of the trees' cache rows: (kv head, slot) -> key, value."""
        kn, vn = ref.to_np(self.k_new), ref.to_np(self.v_new)
        for r in rows:
            n = int(self.n_nodes[r])
            pos = int(self.block_len[self.tree_block[r]]) + ref.depths(self.parent[r], n)
            yield r, n, ref.rotate(kn[r, :n], np.repeat(pos[:, None], self.hkv, 1), self.theta), vn[r, :n]

    def check(self, rows=None, s=None, what=""):
        """Run on outputs filled with a sentinel; every claim of the header."""
        rows = range(self.R) if rows is None else rows
        s = s or self.session()
        k0, v0 = self.k.clone(), self.v.clone()
        out = torch.full((self.R, self.T, self.hq, self.d), 7.0, dtype=TORCH[self.dtype], device="cuda")
        lse = torch.full((self.R, self.T, self.hq), 7.0, device="cuda")
        self.run(s, out, lse)
        torch.cuda.synchronize()
        # 1. the trees' tokens, and nothing else, are written
        touched = torch.zeros(self.cap, dtype=torch.bool, device="cuda")
        ks = 1.0 if self.k_scale is None else ref.to_np(self.k_scale)[:, None]
        vs = 1.0 if self.v_scale is None else ref.to_np(self.v_scale)[:, None]
        sk, sv = self.stored(self.k, self.k_scale), self.stored(self.v, self.v_scale)
        for r, n, key, val in self.expected_tokens(rows):
            at = int(self.tree_start[r])
            touched[at:at + n] = True
            # half a step of the storage type (E4M3: with its subnormal step 2^-10 of the scale, and clipped at
            # 448), and a few fp32 roundings of the rotation: |x0| + |x1| <= 10 times 2^-21
            for got, want, sc in ((sk, key, ks), (sv, val, vs)):
                want = want.transpose(1, 0, 2)
                sc = np.asarray(sc) if self.dtype != "fp8" else sc[:, None]
                if self.dtype == "fp8":
                    want = np.clip(want, -448 * sc, 448 * sc)
                bound = STEP[self.dtype] * np.abs(want) * (1 + 2 ** -10) + 10 * 2.0 ** -21
                if self.dtype == "fp8":
                    bound = bound + 2.0 ** -10 * sc
                assert np.all(np.abs(got[:, at:at + n] - want) <= bound), (what, r)
        for now, before in ((self.k, k0), (self.v, v0)):
            bits, old = now.view(torch.uint8), before.view(torch.uint8)
            assert torch.equal(bits[:, ~touched], old[:, ~touched]), what
        # 2. outputs and lse
        o, l, absv, reach = ref.attend(
            q=ref.to_np(self.q), k=np.nan_to_num(sk), v=np.nan_to_num(sv), block_start=self.block_start,
            block_len=self.block_len, views=self.view_block, offsets=self.view_offset, q_pos=self.q_pos,
            tree_block=self.tree_block, tree_start=self.tree_start,
            n_nodes=np.where(np.isin(np.arange(self.R), list(rows)), self.n_nodes, 0), parent=self.parent,
            heads=self.heads, scale=self.scale, theta=self.theta)
        live = np.zeros((self.R, self.T), bool)
        for r in rows:
            live[r, :self.n_nodes[r]] = True
        got, gl = ref.to_np(out), ref.to_np(lse)
        assert np.all(got[~live] == 7.0) and np.all(gl[~live] == 7.0), what  # left as they were
        assert np.all(np.isfinite(got[live])), what
        err = np.abs(got - o)[live]
        if self.dtype == "f32" or not live.any():
            # fp32 sums of unit-variance values: the library's bar for fp32 storage
            assert not live.any() or (err.max() <= 1e-5 and np.abs(gl - l)[live].max() <= 2e-5), (what, err.max())
            return s, out, lse
        # elementwise: the output's rounding, the weights' rounding (both half a step), and scores that the
        # rounding of the rotated query moves by at most half a step of reach: twice that in a quotient
        step = STEP["bf16"]
        most = step * np.abs(o) + 1.05 * (step + 2 * step * reach[..., None]) * absv + 1e-6
        assert np.all(err <= most[live]), (what, (err / most[live]).max())
        # in the 2-norm roundings are independent and uniform: half a step / sqrt(3) each for the output, the
        # weights, and a score of unit variance (scaled with the scores' spread); 1.5 for the rest
        spread = max(1.0, self.scale * self.d ** 0.5)
        rms = np.sqrt((err ** 2).sum() / (o[live] ** 2).sum())
        assert rms <= 1.5 * step / 3 ** 0.5 * np.sqrt(2 + spread ** 2), (what, rms)
        assert np.abs(gl - l)[live].max() <= (step * reach[live].max() + 1e-4), what
        return s, out, lse


KINDS = [("f32", 64), ("f32", 128), ("bf16", 64), ("bf16", 128), ("fp8", 128)]


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("kind", ["chain", "tree", "forest"])
def test_small_trees(dtype, d, kind):
    Tree(dtype, d=d, kind=kind, seed=3).check()


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("lens", [(0, 0), (1, 0), (0, 1), (1, 1, 1), (63, 64, 65), (127, 128, 129), (255, 16, 257, 112), (2000, 15, 17)])
def test_block_lengths_around_tiles(dtype, d, lens):
    Tree(dtype, d=d, lens=lens, T=3, seed=len(lens)).check()


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 65, 127, 128])
def test_tree_sizes(dtype, d, T):
    Tree(dtype, hq=4, hkv=2, d=d, lens=(200, 30), T=T, seed=T).check()


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (5, 1), (16, 1), (32, 1), (40, 8), (12, 4)])
def test_head_groups(dtype, d, hq, hkv):
    Tree(dtype, hq=hq, hkv=hkv, d=d, lens=(150, 20, 33), T=7, seed=hq).check()


@pytest.mark.parametrize("dtype,d", KINDS)
def test_ragged_trees_and_rows_without_one(dtype, d):
    t = Tree(dtype, d=d, lens=(400, 9, 70, 128, 31), T=20, n_nodes=[20, 0, 1, 13], seed=5)
    t.check()
    Tree(dtype, d=d, lens=(400, 9), T=4, n_nodes=[0], seed=6).check()


@pytest.mark.parametrize("dtype,d", KINDS)
def test_trees_right_behind_their_blocks(dtype, d):
    Tree(dtype, d=d, lens=(90, 40, 128), T=9, in_place=True, seed=8).check()


@pytest.mark.parametrize("dtype,d", KINDS)
def test_permuted_head_map_and_far_positions(dtype, d):
    t = Tree(dtype, hq=12, hkv=3, d=d, lens=(77, 5, 140), T=6, shuffle=True, seed=9, poison=True)
    t.q_pos = t.q_pos + 1_000_000          # rotations by far positions and negative offsets
    t.view_offset = t.view_offset - 37
    t.check()


@pytest.mark.parametrize("dtype,d", KINDS)
def test_views_with_unused_and_repeated_entries(dtype, d):
    vb = [[0, -1, 1, 0], [-1, -1, -1, -1], [2, 2, 2, 2]]
    vo = [[0, 5, 90, 200], [1, 2, 3, 4], [0, 30, 60, 90]]
    Tree(dtype, d=d, lens=(90, 40, 30), views=(vb, vo, [300, 12, 120]), tree_block=[1, 2, 0], T=6, seed=10).check()


@pytest.mark.parametrize("dtype,d", KINDS)
def test_one_block_named_many_times(dtype, d):
    # 64 entries of one row naming one long block: its partial results outnumber one window of the merge
    V = 64
    Tree(dtype, hq=2, hkv=1, d=d, lens=(3000, 4), views=([[0] * V], [list(range(0, 10 * V, 10))], [5000]),
         tree_block=[1], T=2, seed=11).check()


@pytest.mark.parametrize("dtype,d", KINDS)
def test_many_rows_and_short_blocks(dtype, d):
    # more (block, kv head) pairs than CTAs: every CTA crosses many segments
    lens = [40] + [int(x) for x in np.random.default_rng(1).integers(0, 70, 48)]
    Tree(dtype, hq=8, hkv=4, d=d, lens=lens, T=3, seed=12).check(rows=None)


@pytest.mark.parametrize("dtype,d", KINDS)
def test_large_scores_keep_their_order(dtype, d):
    # a softmax scale of 20 / sqrt(D): weights of one nearly everywhere, running maxima that jump
    t = Tree(dtype, d=d, lens=(1000, 50), T=9, seed=13, scale=4.0 * d ** -0.5)
    if dtype == "f32":
        s = t.session()
        out, lse = t.run(s)
        o, l, _, _ = ref.attend(q=ref.to_np(t.q), k=np.nan_to_num(t.stored(t.k, None)), v=np.nan_to_num(t.stored(t.v, None)),
                                block_start=t.block_start, block_len=t.block_len, views=t.view_block,
                                offsets=t.view_offset, q_pos=t.q_pos, tree_block=t.tree_block, tree_start=t.tree_start,
                                n_nodes=t.n_nodes, parent=t.parent, heads=t.heads, scale=t.scale, theta=t.theta)
        # scores of size ~20 in fp32: 20 x 2^-24 x sqrt(D) roundings, twice in a quotient
        assert np.abs(ref.to_np(out) - o).max() <= 4e-5
    else:
        t.check()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp8", 128), ("f32", 128)])
def test_full_size_step(dtype, d):
    # the 40/8-head shape on a long history; rows checked: all heads of two rows' trees
    t = Tree(dtype, hq=40, hkv=8, d=d, lens=(4100, 500, 380, 260, 130), T=24, seed=14, theta=1e6)
    t.check()


def test_same_inputs_same_bits():
    for dtype, d in KINDS:
        t = Tree(dtype, hq=8, hkv=2, d=d, lens=(900, 100, 50), T=12, n_nodes=[12, 8], seed=15)
        s = t.session()
        o1, l1 = t.run(s)
        o1, l1 = o1.clone(), l1.clone()
        o2, l2 = t.run(s)
        live = torch.zeros(2, 12, dtype=torch.bool, device="cuda")
        live[0, :12] = live[1, :8] = True
        assert torch.equal(o1[live], o2[live]) and torch.equal(l1[live], l2[live])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_a_chain_is_a_query_chunk(dtype):
    """A chain's tokens, counted into the block, are what a chunk of queries
    with view limits attends: two paths of the library, one result."""
    T = 6
    t = Tree(dtype, hq=10, hkv=2, lens=(500, 60, 33), T=T, kind="chain", in_place=True, seed=16, poison=False)
    out, lse = t.run(t.session())
    lens2 = t.block_len + np.asarray([0, T, T], np.int32)
    # every row of a worker's chunk sees the other worker's block as the tree's rows do: without its tree
    vb, vo, vl, qp = api.views_chunked("combined", lens2, 1, 2, T)
    vl = np.where(vb == 0, -1, vl)
    for w in range(2):
        for i in range(T):
            r = w * T + i
            for v in range(3):
                b = vb[r, v]
                vo[r, v] = t.view_offset[w][list(t.view_block[w]).index(b)]
                if b == 2 - w:
                    vl[r, v] = t.block_len[b]
            qp[r] = t.q_pos[w] + i
    s = engine.DecodeSession(n_rows=2 * T, n_q_heads=10, n_kv_heads=2, head_dim=128, n_blocks=3, max_view_blocks=3,
                             capacity=t.cap, dtype=torch.bfloat16, rope_theta=t.theta, view_limits=True,
                             kv_fp8=dtype == "fp8")
    s.set_metadata(t.block_start, lens2, vb, vo, qp)
    s.plan_limited(vl)
    q = t.q.reshape(2 * T, 10, 128)
    if dtype == "fp8":
        o2, l2 = s.decode_planned_fp8(q, t.k.view(torch.uint8), t.v.view(torch.uint8), t.k_scale, t.v_scale)
    else:
        o2, l2 = s.decode_planned(q, t.k, t.v)
    a, b = ref.to_np(out).reshape(2 * T, 10, 128), ref.to_np(o2)
    # both round the output (half a step each) and the weights; scores differ by the query's rounding
    assert np.sqrt(((a - b) ** 2).sum() / (b ** 2).sum()) <= 1.5 * 2.0 ** -8 / 3 ** 0.5 * 5 ** 0.5
    assert np.abs(ref.to_np(lse).reshape(2 * T, 10) - ref.to_np(l2)).max() <= 2e-2


# ------------------------------------------------------------------ refusals

def flags_of(t, **change):
    for key, val in change.items():
        setattr(t, key, np.asarray(val, np.int32))
    s = t.session()
    return s, s.device_flags()


def test_bad_rows_are_reported_and_left_out():
    base = dict(lens=(100, 20, 30, 40), T=4, seed=20)
    for what, change, bit in (
            ("too many nodes", dict(n_nodes=[4, 5, 4]), 64), ("negative nodes", dict(n_nodes=[4, -1, 4]), 64),
            ("a parent after its child", dict(parent=[[-1, 0, 1, 2], [-1, 2, 0, 1], [-1, 0, 0, 0]]), 64),
            ("its own parent", dict(parent=[[-1, 0, 1, 2], [-1, 1, 0, 1], [-1, 0, 0, 0]]), 64),
            ("a parent below -1", dict(parent=[[-1, 0, 1, 2], [-2, 0, 0, 1], [-1, 0, 0, 0]]), 64),
            ("no block", dict(tree_block=[1, -1, 3]), 1), ("a block past the table", dict(tree_block=[1, 4, 3]), 1)):
        t = Tree("bf16", **base)
        s, f = flags_of(t, **change)
        assert f == bit, what
        t.tree_block = np.clip(t.tree_block, 0, 3)
        t.n_nodes = np.clip(t.n_nodes, 0, 4)
        t.parent[1] = [-1, 0, 0, 0]
        t.check(rows=[0, 2], s=s, what=what)


def test_trees_that_meet_other_tokens_are_reported_and_left_out():
    for what, at in (("a block", lambda t: t.block_start[2] + 29), ("its own block", lambda t: t.block_start[2] + 3),
                     ("past the pool", lambda t: t.cap - 3), ("before the pool", lambda t: -1)):
        t = Tree("bf16", lens=(100, 20, 30, 40), T=4, seed=21)
        ts = t.tree_start.copy()
        ts[1] = at(t)
        s, f = flags_of(t, tree_start=ts)
        assert f == 2, what
        t.check(rows=[0, 2], s=s, what=what)
    t = Tree("bf16", lens=(100, 20, 30, 40), T=4, seed=21)
    ts = t.tree_start.copy()
    ts[1] = ts[0] + 3
    s, f = flags_of(t, tree_start=ts)
    assert f == 2
    t.check(rows=[2], s=s)


def test_bad_blocks_and_views_are_skipped():
    t = Tree("bf16", lens=(100, 20, 30), T=4, seed=22)
    good = t.block_len.copy()
    s, f = flags_of(t, view_block=[[0, 7, 1], [0, 1, 2]])
    assert f == 1
    t.view_block = np.asarray([[0, -1, 1], [0, 1, 2]], np.int32)
    t.check(s=s)
    t = Tree("bf16", lens=(100, 20, 30), T=4, seed=22)
    s, f = flags_of(t, block_len=[t.cap + 1, 20, 30])
    assert f == 2
    t.block_len = np.asarray([0, 20, 30], np.int32)
    t.check(s=s)
    assert good[1] == 20


def test_unequal_head_groups_leave_every_row_out():
    t = Tree("bf16", hq=4, hkv=2, lens=(50, 10), T=3, shuffle=True, seed=23)
    s, f = flags_of(t, heads=[0, 0, 0, 1])
    assert f == 4
    t.check(rows=[], s=s)


def test_a_missing_or_other_plan_is_reported():
    t = Tree("bf16", lens=(50, 10), T=3, seed=24)
    s = t.session()
    api.workspace_init(s.workspace, s.ws_bytes)
    t.check(rows=[], s=s)
    assert s.device_flags() == 32
    path = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    s.commit(t.k, t.v, path, torch.ones(1, dtype=torch.int32, device="cuda"))
    assert s.device_flags() == 32


# ------------------------------------------------------------- verification

def draw_verify(rng, R, T, V, dtype, drawn, branch="tree", n_nodes=None, alike=0.7):
    n_nodes = np.full(R, T, np.int32) if n_nodes is None else np.asarray(n_nodes, np.int32)
    parent = ref.random_parents(rng, R, T, branch, np.maximum(0, np.minimum(n_nodes, T)))
    logits = 2 * rng.standard_normal((R, T, V))
    p = np.exp(logits)
    q = np.exp(logits + alike * rng.standard_normal((R, T, V)))
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    p = torch.tensor(p / p.sum(-1, keepdims=True)).to(dt)
    q = torch.tensor(q / q.sum(-1, keepdims=True)).to(dt)
    token = np.zeros((R, T), np.int32)
    for r in range(R):
        for i in range(1, T):
            w = q[r, max(0, parent[r, i])].double().numpy()
            token[r, i] = rng.choice(V, p=w / w.sum()) if drawn else int(np.argsort(-w, kind="stable")[min(V - 1, int(rng.integers(0, 3)))])
    return dict(n_nodes=n_nodes, parent=parent, token=token, p=p, q=q if drawn else None,
                u_accept=rng.random((R, T), dtype=np.float32), u_sample=rng.random(R, dtype=np.float32))


def run_verify(x, p=None, q=None):
    p = x["p"].cuda() if p is None else p
    q = (None if x["q"] is None else x["q"].cuda()) if q is None else q
    got = engine.tree_verify(ref.dev(x["n_nodes"]), ref.dev(x["parent"]), ref.dev(x["token"]), p, q,
                             ref.dev(x["u_accept"], torch.float32), ref.dev(x["u_sample"], torch.float32))
    return [g.cpu().numpy() for g in got]


def check_verify(x, **kw):
    path, n_path, nxt = run_verify(x, **kw)
    for r in range(len(x["n_nodes"])):
        want = ref.verify(x["n_nodes"][r], x["parent"][r], x["token"][r], x["p"][r].float().numpy(),
                          None if x["q"] is None else x["q"][r].float().numpy(), x["u_accept"][r], x["u_sample"][r])
        assert (list(path[r]), int(n_path[r]), int(nxt[r])) == (list(want[0]), want[1], want[2]), r


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V", [1, 2, 3, 5, 100, 127, 128, 129, 1000, 4097, 50021])
def test_verify_vocabularies(dtype, drawn, V):
    rng = np.random.Generator(np.random.PCG64(V))
    check_verify(draw_verify(rng, 6, 7, V, dtype, drawn))


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("T,branch", [(1, "chain"), (2, "chain"), (16, "chain"), (40, "forest"), (128, "tree")])
def test_verify_trees(drawn, T, branch):
    rng = np.random.Generator(np.random.PCG64(T))
    check_verify(draw_verify(rng, 5, T, 211, "f32", drawn, branch, alike=0.3))
    check_verify(draw_verify(rng, 4, T, 211, "f32", drawn, branch, n_nodes=[T, 0, 1, T // 2 + 1]))


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_many_rejections_at_one_node(drawn):
    # a star: every child of the root tested in turn against what is left
    rng = np.random.Generator(np.random.PCG64(3))
    x = draw_verify(rng, 8, 64, 500, "f32", drawn)
    x["parent"][:, 1:] = 0
    x["u_accept"][:] = np.float32(1 - 2.0 ** -24)  # rejected whenever it can be
    check_verify(x)
    x["token"][:, 2::2] = x["token"][:, 1:-1:2]   # the same token twice
    check_verify(x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 1, 2, 3, 8])
def test_verify_strided_rows(dtype, pad):
    rng = np.random.Generator(np.random.PCG64(pad))
    x = draw_verify(rng, 4, 9, 333, dtype, True)
    p = torch.full((4, 9, 333 + pad), 9.0, dtype=x["p"].dtype, device="cuda")
    q = torch.full((4, 9, 333 + 5), 9.0, dtype=x["p"].dtype, device="cuda")
    p[..., :333], q[..., 5:] = x["p"], x["q"]
    check_verify(x, p=p[..., :333], q=q[..., 5:])


def test_verify_edges():
    rng = np.random.Generator(np.random.PCG64(4))
    x = draw_verify(rng, 7, 6, 50, "f32", True, "chain")
    x["q"] = x["p"].clone()                 # drafts from the target itself: all stand
    x["u_accept"][:] = np.float32(1 - 2.0 ** -24)
    path, n_path, _ = run_verify(x)
    assert np.all(n_path == 6)
    check_verify(x)
    x["p"][0] = 0                            # nothing to accept, nothing to draw
    x["p"][1] = 0
    x["p"][1, :, 7] = 1                      # one certain token
    x["p"][2, :, 3] = float("nan")           # NaN and negative values count as 0, larger ones as 1
    x["p"][2, :, 4] = -1
    x["p"][2, :, 5] = float("inf")
    x["q"][3] = 0                            # a draft that could not have been drawn
    x["u_accept"][4] = 0                     # everything possible stands
    x["u_sample"][4] = 0
    x["u_sample"][5] = np.float32(1 - 2.0 ** -24)
    check_verify(x)


def test_verify_refuses_bad_rows_alone():
    rng = np.random.Generator(np.random.PCG64(5))
    x = draw_verify(rng, 7, 6, 50, "f32", True)
    x["n_nodes"][0], x["n_nodes"][1] = 7, -1
    x["parent"][2, 3] = 3
    x["token"][3, 2] = 50
    x["token"][4, 5] = -1
    x["token"][5, 0] = -7                    # the root's token is not used
    path, n_path, nxt = run_verify(x)
    assert list(n_path[:5]) == [0] * 5 and list(nxt[:5]) == [-1] * 5 and np.all(path[:5] == -1)
    assert np.all(n_path[5:] >= 1)
    check_verify(x)


@pytest.mark.parametrize("drawn", [True, False])
def test_verified_tokens_follow_the_target(drawn):
    """Drafts or not, the first token after the root has the target's law."""
    rng = np.random.Generator(np.random.PCG64(6))
    V, R, rounds = 6, 4096, 4
    p = rng.dirichlet(np.ones(V))
    q = rng.dirichlet(np.ones(V))
    count = np.zeros(V)
    for _ in range(rounds):
        token = np.zeros((R, 4), np.int32)
        token[:, 1:] = rng.choice(V, size=(R, 3), p=q) if drawn else np.argsort(-q)[:3]
        x = dict(n_nodes=np.full(R, 4), parent=np.tile([-1, 0, 0, 0], (R, 1)), token=token,
                 p=torch.tensor(np.tile(p, (R, 4, 1))).float(),
                 q=torch.tensor(np.tile(q, (R, 4, 1))).float() if drawn else None,
                 u_accept=rng.random((R, 4), dtype=np.float32), u_sample=rng.random(R, dtype=np.float32))
        path, n_path, nxt = run_verify(x)
        first = np.where(n_path > 1, token[np.arange(R), np.maximum(path[:, 1], 0)], nxt)
        count += np.bincount(first, minlength=V)
    n = R * rounds
    sigma = np.sqrt(p * (1 - p) / n)
    assert np.all(np.abs(count / n - p) <= 5 * sigma + 1e-6)  # five standard deviations, seeded


# ------------------------------------------------------------------- commit

@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("layers", [1, 5])
def test_commit_moves_the_path(dtype, d, in_place, layers):
    T = 40
    t = Tree(dtype, hq=4, hkv=2, d=d, lens=(50, 7, 30, 64, 5), T=T, n_nodes=[40, 40, 0, 11], in_place=in_place, seed=30)
    s = t.session()
    paths = [[0, 1, 2, 5, 9, 17, 38, 39], list(range(40)), [], [10]]
    path = np.full((4, T), -1, np.int32)
    for r, x in enumerate(paths):
        path[r, :len(x)] = x
    g = torch.Generator(device="cuda").manual_seed(1)
    shape = (layers, 2, t.cap, d)
    k = torch.randn(shape, generator=g, device="cuda").to(t.k.dtype)
    v = torch.randn(shape, generator=g, device="cuda").to(t.k.dtype)
    want = [x.clone().view(torch.uint8) for x in (k, v)]
    for x in want:
        for r, line in enumerate(paths):
            end = int(t.block_start[r + 1] + t.block_len[r + 1])
            src = [int(t.tree_start[r]) + i for i in line]
            x[:, :, end:end + len(line)] = x[:, :, src].clone()
    s.commit(k if layers > 1 else k[0], v if layers > 1 else v[0], ref.dev(path), ref.dev([len(x) for x in paths]))
    assert s.device_flags() == 0
    assert torch.equal(k.view(torch.uint8), want[0]) and torch.equal(v.view(torch.uint8), want[1])


def test_commit_refuses_bad_paths_and_places():
    def run(path, n_path, bit, **kw):
        t = Tree("bf16", hq=4, hkv=2, lens=(50, 7, 30), T=4, seed=31, **kw)
        s = t.session()
        k, v = t.k.clone(), t.v.clone()
        s.commit(k, v, ref.dev(path), ref.dev(n_path))
        assert s.device_flags() == bit
        # row 0 moves nothing, row 1 its token 0 and 2
        end = int(t.block_start[2] + t.block_len[2])
        want = t.k.clone()
        want[:, end:end + 2] = want[:, [int(t.tree_start[1]), int(t.tree_start[1]) + 2]]
        assert torch.equal(k.view(torch.int16), want.view(torch.int16))
    ok = [0, 2, -1, -1]
    run([[0, 0, 1, 1], ok], [2, 2], 64)
    run([[1, 0, 1, 1], ok], [2, 2], 64)
    run([[0, 4, 1, 1], ok], [2, 2], 64)
    run([[-1, 0, 1, 1], ok], [2, 2], 64)
    run([[0, 1, 2, 3], ok], [5, 2], 64)
    run([[0, 1, 2, 3], ok], [-1, 2], 64)
    run([[0, 1, 2, 3], ok], [0, 2], 0)
    run([[2, 3, -1, -1], ok], [2, 2], 64, n_nodes=[3, 4])
    # blocks without a gap: the path would run into the next block, or past the pool
    t = Tree("bf16", hq=4, hkv=2, lens=(50, 7, 30), T=4, seed=31)
    t.block_start = np.asarray([0, 60, 69], np.int32)
    s = t.session()
    s.commit(t.k, t.v, ref.dev([[0, 1, 2, 3], ok]), ref.dev([3, 2]))
    assert s.device_flags() == 2
    t = Tree("bf16", hq=4, hkv=2, lens=(50, 7, 30), T=4, seed=31)
    t.block_start = np.asarray([0, t.cap - 8, 60], np.int32)
    t.tree_start = np.asarray([100, 110], np.int32)  # (the pool has 130 tokens)
    s = t.session()
    assert s.device_flags() == 0
    s.commit(t.k, t.v, ref.dev([[0, 1, 2, 3], ok]), ref.dev([2, 2]))
    assert s.device_flags() == 2


# ----------------------------------------------------------------- together

def speculative_step(t, s, x, layers, out, stream=None):
    """Decode every layer, verify, commit: what a serving loop does."""
    for l in range(len(layers)):
        k, v = layers[l]
        s.decode(t.q, t.k_new, t.v_new, k, v, out=out[l], want_lse=False, stream=stream)
    return engine.tree_verify(*x, stream=stream)


def make_run(seed=40):
    t = Tree("bf16", hq=10, hkv=2, lens=(260, 40, 33), T=6, in_place=True, seed=seed)
    rng = np.random.Generator(np.random.PCG64(seed))
    x = draw_verify(rng, t.R, t.T, 1000, "f32", True, n_nodes=t.n_nodes)
    x["parent"] = t.parent
    args = [ref.dev(x["n_nodes"]), ref.dev(x["parent"]), ref.dev(x["token"]), x["p"].cuda(), x["q"].cuda(),
            ref.dev(x["u_accept"], torch.float32), ref.dev(x["u_sample"], torch.float32)]
    return t, x, args


def test_a_step_and_the_next():
    """Two steps in a row: the second attends the first's accepted tokens."""
    t, x, args = make_run()
    L = 3
    g = torch.Generator(device="cuda").manual_seed(2)
    kp = torch.stack([t.k] + [torch.randn(t.k.shape, generator=g, device="cuda").to(t.k.dtype) for _ in range(L - 1)])
    vp = torch.stack([t.v] + [torch.randn(t.v.shape, generator=g, device="cuda").to(t.v.dtype) for _ in range(L - 1)])
    s = t.session()
    out = [torch.empty_like(t.q) for _ in range(L)]
    path, n_path, nxt = speculative_step(t, s, args, [(kp[l], vp[l]) for l in range(L)], out)
    s.commit(kp, vp, path, n_path)
    assert s.device_flags() == 0
    # the next step's metadata; one new root a row
    grown = n_path.cpu().numpy()
    t2 = Tree("bf16", hq=10, hkv=2, lens=tuple(t.block_len + np.concatenate([[0], grown])), T=1, in_place=True, seed=41)
    t2.block_start = t.block_start.copy()
    t2.tree_start = (t2.block_start + t2.block_len)[t2.tree_block]
    t2.cap, t2.k, t2.v = t.cap, kp[0], vp[0]
    # the cache holds the accepted tokens at their positions
    kn = ref.to_np(t.k_new)
    for r in range(t.R):
        line = path[r, :grown[r]].cpu().numpy()
        assert list(ref.depths(t.parent[r], t.T)[line]) == list(range(grown[r]))
        end = int(t.block_start[r + 1] + t.block_len[r + 1])
        want = ref.rotate(kn[r, line], np.repeat((t.block_len[r + 1] + np.arange(grown[r]))[:, None], 2, 1), t.theta)
        got = ref.to_np(kp[0][:, end:end + grown[r]]).transpose(1, 0, 2)
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) * (1 + 2 ** -10) + 1e-5)
    t2.check()


def test_captured_step_replays_on_new_inputs():
    t, x, args = make_run(42)
    s = t.session()
    out = [torch.empty_like(t.q)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    path = torch.full((t.R, t.T), -9, dtype=torch.int32, device="cuda")
    n_path = torch.zeros(t.R, dtype=torch.int32, device="cuda")
    nxt = torch.zeros(t.R, dtype=torch.int32, device="cuda")
    kp, vp = t.k.clone(), t.v.clone()
    with torch.cuda.stream(st):
        s.plan(ref.dev(t.tree_block), ref.dev(t.n_nodes), ref.dev(t.parent))
    trees = s.trees
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        api.attn_plan_tree(s.desc, t.T, *s.meta, *trees, s.workspace, s.ws_bytes)
        s.decode(t.q, t.k_new, t.v_new, kp, vp, out=out[0], want_lse=False)
        engine.tree_verify(*args, path=path, n_path=n_path, next_token=nxt)
        s.commit(kp, vp, path, n_path)
    for seed in (43, 44):
        t2, x2, args2 = make_run(seed)
        for a, b in zip(args, args2):
            a.copy_(b)
        trees[2].copy_(ref.dev(t2.parent))
        t.q.copy_(t2.q)
        t.k_new.copy_(t2.k_new)
        t.v_new.copy_(t2.v_new)
        kp.copy_(t2.k)
        vp.copy_(t2.v)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        s2 = t2.session()
        o2 = torch.empty_like(t2.q)
        s2.decode(t2.q, t2.k_new, t2.v_new, t2.k, t2.v, out=o2, want_lse=False)
        p2, n2, x2 = engine.tree_verify(*args2)
        s2.commit(t2.k, t2.v, p2, n2)
        assert torch.equal(out[0], o2) and torch.equal(path, p2) and torch.equal(n_path, n2) and torch.equal(nxt, x2)
        assert torch.equal(kp.view(torch.int16), t2.k.view(torch.int16))
        assert torch.equal(vp.view(torch.int16), t2.v.view(torch.int16))
    assert s.device_flags() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp8", 128), ("f32", 64)])
def test_two_sessions_on_two_streams(dtype, d):
    a = Tree(dtype, hq=8, hkv=2, d=d, lens=(3000, 100, 50), T=12, seed=50)
    b = Tree(dtype, hq=8, hkv=2, d=d, lens=(2500, 10, 500), T=9, seed=51)
    want = []
    for t in (a, b):
        o, l = t.run(t.session())
        want.append((o.clone(), l.clone()))
    sessions = [a.session(), b.session()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(4):
        for i, t in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i] = t.run(sessions[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])


def test_outputs_at_any_element_address():
    for dtype, d in (("bf16", 128), ("f32", 64)):
        t = Tree(dtype, hq=4, hkv=2, d=d, lens=(70, 11), T=3, seed=52)
        s = t.session()
        o1, l1 = t.run(s)
        buf = torch.zeros(o1.numel() + 1, dtype=o1.dtype, device="cuda")
        o2 = buf[1:].view(o1.shape)
        t.run(s, o2, l1)
        assert torch.equal(o1, o2) and float(buf[0]) == 0


# ------------------------------------------------------- values, views, sizes

def bits(x):
    return x.contiguous().view(torch.uint8)


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("where", ["v_new", "k_new", "v", "k", "q"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_stay_with_their_readers(dtype, d, where, value):
    """Queries that do not attend such a token give the same bits as without
    it; those that do are not finite."""
    def make():
        return Tree(dtype, hq=6, hkv=2, d=d, lens=(200, 40, 130), views=([[0, 1], [0, 2]], [[0, 200], [0, 200]], [240, 330]),
                    T=7, kind="forest", seed=60)
    clean, t = make(), make()
    o0, l0 = clean.run(clean.session())
    touched = torch.zeros(t.R, t.T, t.hq, dtype=torch.bool, device="cuda")
    G = t.hq // t.hkv
    if where in ("v_new", "k_new"):   # row 0's node 2, kv head 1
        getattr(t, where)[0, 2, 1, 5] = value
        anc = ref.ancestors(t.parent[0], t.T)
        for i in range(t.T):
            touched[0, i, G:] = bool(anc[i, 2])
    elif where == "q":
        t.q[1, 3, 4, 9] = value
        touched[1, 3, 4] = True
    else:                             # block 2, which row 0 does not see
        getattr(t, where)[0, int(t.block_start[2]) + 5, 7] = value if dtype != "fp8" else float("nan")
        touched[1, :, :G] = True
    o1, l1 = t.run(t.session())
    assert torch.equal(bits(o1[~touched]), bits(o0[~touched])) and torch.equal(l1[~touched], l0[~touched])
    stored_as_448 = dtype == "fp8" and where in ("v_new", "k_new") and value == value
    # (an infinite score of -inf is a token without weight)
    if not stored_as_448 and not (value != value) and where in ("k_new", "k"):
        return
    if not stored_as_448:
        assert not torch.isfinite(o1[touched].float()).all(-1).any()


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("power", [-30, 20])
def test_scaled_queries(dtype, d, power):
    """Powers of two that move from the queries to the softmax scale."""
    t = Tree(dtype, hq=6, hkv=2, d=d, lens=(150, 40), T=5, seed=61)
    o1, l1 = t.run(t.session())
    o1, l1 = o1.clone(), l1.clone()
    t.q = t.q * 2.0 ** power
    t.scale = t.scale * 2.0 ** -power
    o2, l2 = t.run(t.session())
    assert torch.equal(bits(o1), bits(o2)) and torch.equal(l1, l2)


@pytest.mark.parametrize("dtype,d", KINDS)
def test_queries_of_zero(dtype, d):
    t = Tree(dtype, hq=6, hkv=2, d=d, lens=(150, 40), T=5, seed=62)
    t.q.zero_()
    t.check()


@pytest.mark.parametrize("dtype,d", KINDS)
def test_wide_and_narrow_groups_in_turn(dtype, d):
    # 700, 42 and 350 columns a kv head: full groups of queries and rests, for one CTA or more each
    Tree(dtype, hq=14, hkv=2, d=d, lens=(700, 60, 33, 129), T=100, n_nodes=[100, 6, 50], seed=63).check()
    Tree(dtype, hq=14, hkv=2, d=d, lens=(9000, 60, 33, 129), T=50, n_nodes=[50, 6, 21], seed=64).check(what="long")


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("seed", [65, 66, 67])
def test_rows_with_views_of_their_own(dtype, d, seed):
    rng = np.random.Generator(np.random.PCG64(seed))
    B, R, V = 9, 12, 5
    lens = [int(x) for x in rng.integers(0, 300, B)]
    vb = rng.integers(-1, B, (R, V))
    vo = rng.integers(0, 2000, (R, V))
    Tree(dtype, hq=4, hkv=2, d=d, lens=lens, views=(vb, vo, rng.integers(500, 3000, R)),
         tree_block=rng.integers(0, B, R), n_nodes=rng.integers(0, 12, R), T=11, seed=seed).check()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp8", 128), ("f32", 64)])
def test_hundreds_of_rows(dtype, d):
    # (two rows a block: HW_MAX_BLOCKS is 256)
    lens = [30] + [int(x) for x in np.random.default_rng(2).integers(0, 9, 250)]
    own = 1 + np.arange(500) % 250
    Tree(dtype, hq=2, hkv=1, d=d, lens=lens, views=([[0, b] for b in own], [[0, 30]] * 500, [31] * 500), tree_block=own, T=2,
         seed=68).check()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp8", 128), ("f32", 128)])
def test_offsets_past_32_bits(dtype, d):
    """The same tokens in a small pool and at the end of one whose elements
    pass 2^32: the same bits."""
    t = Tree(dtype, hq=4, hkv=2, d=d, lens=(300, 40, 129), T=6, seed=69, poison=False)
    o1, l1 = t.run(t.session())
    o1, l1 = o1.clone(), l1.clone()
    small = t.k.clone(), t.v.clone()
    end = 2 ** 32 // (2 * d) + 1000    # tokens of a head; two heads
    move = end - t.cap
    big = torch.zeros(2, 2, end, d, dtype=t.k.dtype, device="cuda")
    big[0, :, move:], big[1, :, move:] = t.k, t.v
    for r in range(t.R):               # without the trees' tokens
        big[:, :, move + int(t.tree_start[r]):move + int(t.tree_start[r]) + t.T] = 0
    t.k, t.v, t.cap = big[0], big[1], end
    t.block_start, t.tree_start = t.block_start + move, t.tree_start + move
    s = t.session()
    o2, l2 = t.run(s)
    assert torch.equal(bits(o1), bits(o2)) and torch.equal(l1, l2)
    assert torch.equal(bits(t.k[:, move:]), bits(small[0])) and torch.equal(bits(t.v[:, move:]), bits(small[1]))
    assert int(bits(t.k[:, :move]).max()) == 0
    # an accepted path moves there too
    path = np.full((t.R, t.T), -1, np.int32)
    path[:, :2] = [0, 3]
    s.commit(t.k, t.v, ref.dev(path), ref.dev([2] * t.R))
    assert s.device_flags() == 0
    for r in range(t.R):
        at, src = int(t.block_start[r + 1] + t.block_len[r + 1]), int(t.tree_start[r])
        for j, i in enumerate((0, 3)):
            assert torch.equal(bits(t.k[:, at + j]), bits(t.k[:, src + i]))
            assert torch.equal(bits(t.v[:, at + j]), bits(t.v[:, src + i]))


@pytest.mark.parametrize("R", [3, 25])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("drawn", [True, False])
def test_verify_long_vocabularies(R, dtype, drawn):
    # few rows: sixteen CTAs each; many: eight; the longer vocabulary is read again at every step
    for V in (150_001, 1_500_000 if R == 3 else 700_000):
        rng = np.random.Generator(np.random.PCG64(V))
        T = 3
        w = rng.random((R, T, V), dtype=np.float32) ** 8
        p = torch.tensor(w / w.sum(-1, keepdims=True))
        w *= rng.random((R, T, V), dtype=np.float32) + 0.5
        q = torch.tensor(w / w.sum(-1, keepdims=True))
        dt = torch.float32 if dtype == "f32" else torch.bfloat16
        # (the likeliest of 64 tokens: what is below 2^-56 counts as 0, and was not drawn either)
        some = rng.integers(0, V, (R, T, 64))
        token = np.take_along_axis(some, np.take_along_axis(w[:, :1].repeat(T, 1), some, 2).argmax(2)[..., None], 2)[..., 0].astype(np.int32)
        x = dict(n_nodes=np.full(R, T), parent=np.tile([-1, 0, 0], (R, 1)), token=token, p=p.to(dt), q=q.to(dt) if drawn else None, u_accept=rng.random((R, T), dtype=np.float32),
                 u_sample=rng.random(R, dtype=np.float32))
        check_verify(x)


def test_sessions_that_share_a_pool_and_a_stream():
    """Two plans in turn on one pool, as two groups of workers would have:
    neither disturbs the other's blocks."""
    a = Tree("bf16", hq=4, hkv=2, lens=(300, 40, 129), T=6, seed=70)
    b = Tree("bf16", hq=4, hkv=2, lens=(90, 200), T=4, seed=71)
    pool_k = torch.cat([a.k, b.k], 1).contiguous()
    pool_v = torch.cat([a.v, b.v], 1).contiguous()
    b.block_start, b.tree_start = b.block_start + a.cap, b.tree_start + a.cap
    a.cap = b.cap = a.cap + b.cap
    for t in (a, b):
        t.k, t.v = pool_k, pool_v
    sa, sb = a.session(), b.session()
    b.check(s=sb)
    a.check(s=sa)
    b.check(s=sb)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp8", 128), ("f32", 64)])
def test_the_largest_description(dtype, d):
    """HW_MAX_VIEW_ENTRIES rows and HW_MAX_TREE_QUERIES nodes, HW_MAX_BLOCKS blocks."""
    R, B = 4096, 256
    rng = np.random.Generator(np.random.PCG64(72))
    own = np.arange(R) % B
    Tree(dtype, hq=1, hkv=1, d=d, lens=[int(x) for x in rng.integers(0, 40, B)], views=(own[:, None], np.zeros((R, 1)), rng.integers(0, 99, R)),
         tree_block=own, n_nodes=rng.integers(0, 17, R), T=16, seed=72).check()


def test_the_longest_verification():
    # HW_MAX_VOCAB values, bf16: a row's slices fit no shared memory
    V = 1 << 24
    g = torch.Generator(device="cuda").manual_seed(3)
    p = torch.rand(1, 2, V, generator=g, device="cuda").pow(40).bfloat16()
    p = (p.float() / p.float().sum(-1, keepdim=True)).bfloat16()
    token = p[0, 0].float().topk(2).indices.int()
    x = dict(n_nodes=np.array([2]), parent=np.array([[-1, 0]]), token=token.cpu().numpy()[None].astype(np.int32), p=p.cpu(), q=None,
             u_accept=np.full((1, 2), 0.999, np.float32), u_sample=np.array([0.37], np.float32))
    check_verify(x)


# ------------------------------------------------------- many clusters at once

@pytest.mark.parametrize("dtype,V", [("f32", 2003), ("bf16", 40_001), ("f32", 300_000)])
@pytest.mark.parametrize("drawn", [True, False])
def test_verify_more_rows_than_run_at_once(dtype, V, drawn):
    """Clusters that start as others end, rows that leave at once between those
    that exchange sums, slices that leave room for one CTA an SM (the longest
    vocabulary, nine rows: sixteen CTAs each): every row as by itself."""
    R = 9 if V == 300_000 else 250
    rng = np.random.Generator(np.random.PCG64(V))
    n = rng.integers(-1, 6, R) if R > 9 else np.array([4, 0, 3, 5, 4, 2, 1, 4, 3])  # (-1 and 5 are refused)
    x = draw_verify(rng, R, 4, V if R == 9 else 64, dtype, drawn, n_nodes=n)
    if R > 9:  # the values spread over the vocabulary: p and q of 64 tokens, 0 elsewhere
        at = np.sort(rng.choice(V, 64, replace=False))
        wide = {k: torch.zeros(R, 4, V, dtype=x[k].dtype) for k in ("p", "q") if x[k] is not None}
        for k, t in wide.items():
            t[..., torch.as_tensor(at)] = x[k]
        x.update(wide, token=at[x["token"]].astype(np.int32))
    for _ in range(3):
        check_verify(x)


# ------------------------------------------- turns of the two streams of a CTA

@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T", [4, 50])
@pytest.mark.parametrize("seed", [80, 81, 82])
def test_groups_of_odd_numbers_of_tiles(dtype, T, seed):
    """Many groups behind one another in a CTA, of one to some tiles each, so
    that groups end with either stream; of up to 128 queries and of more in
    turn.  Repeated runs give the same bits."""
    rng = np.random.Generator(np.random.PCG64(seed))
    R = 48
    # every row's own block alone: a group a row; 8 queries a node, so 50 nodes fill more than one query tile
    lens = [int(x) for x in rng.choice([1, 100, 128, 129, 300, 384, 500, 640, 1100], R)]
    n = rng.integers(1, T + 1, R)
    t = Tree(dtype, hq=32, hkv=4, lens=lens, views=([[b] for b in range(R)], [[0]] * R, lens), tree_block=np.arange(R), T=T,
             n_nodes=n, seed=seed)
    s, out, lse = t.check(what="odd")
    live = torch.as_tensor(np.arange(T)[None] < n[:, None]).cuda()
    for _ in range(20):
        o2, l2 = t.run(s)
        assert torch.equal(bits(o2[live]), bits(out[live])) and torch.equal(l2[live], lse[live])
    assert s.device_flags() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("seed", [83, 84])
def test_narrow_groups_in_ctas_with_a_wide_one(dtype, seed):
    """Groups of over 128 queries and groups of few with many tiles, row by
    row: every stage of either ring is used again and again."""
    rng = np.random.Generator(np.random.PCG64(seed))
    R = 12
    lens = [int(x) for x in rng.choice([20, 2100, 5000, 9001], R)]
    n = np.where(np.arange(R) % 3 == 0, 40, rng.integers(1, 5, R))
    t = Tree(dtype, hq=16, hkv=4, lens=lens, views=([[b] for b in range(R)], [[0]] * R, lens), tree_block=np.arange(R), T=40,
             n_nodes=n, seed=seed)
    s, out, lse = t.check(what="wide and narrow")
    live = torch.as_tensor(np.arange(40)[None] < n[:, None]).cuda()
    for _ in range(20):
        o2, l2 = t.run(s)
        assert torch.equal(bits(o2[live]), bits(out[live])) and torch.equal(l2[live], lse[live])
    assert s.device_flags() == 0


@pytest.mark.parametrize("mass", [3.0, 64.0, 120.0, 127.5, 128.0])
def test_verify_rows_whose_sum_is_not_one(mass):
    """A row of p may sum to 128: c grows by up to that much a rejection."""
    rng = np.random.Generator(np.random.PCG64(int(2 * mass)))
    R, T, V = 64, 128, 300
    p = np.zeros((R, T, V), np.float32)
    q = np.zeros((R, T, V), np.float32)
    p[:, 0, :128] = np.float32(mass / 128)
    # tokens 200 .. 249 cannot stand; a few others can while c q is below p
    q[:, 0, 200:250] = np.float32(0.01)
    some = rng.integers(0, 128, (R, 8))
    for r in range(R):
        q[r, 0, some[r]] = np.float32(2.0) ** -rng.integers(7, 16, 8) * rng.random(8, dtype=np.float32)
    p[:, 1:, 5] = 1
    q[:, 1:, 6] = 1
    token = rng.integers(200, 250, (R, T)).astype(np.int32)
    late = rng.integers(2, 10, R)          # rejections before the first that could stand
    for r in range(R):
        token[r, late[r]::3] = rng.choice(some[r], len(token[r, late[r]::3]))
    x = dict(n_nodes=rng.integers(2, T + 1, R), parent=np.tile(np.r_[-1, np.zeros(T - 1)], (R, 1)).astype(np.int32), token=token,
             p=torch.tensor(p), q=torch.tensor(q), u_accept=rng.random((R, T), dtype=np.float32), u_sample=rng.random(R, dtype=np.float32))
    check_verify(x)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V", [1000, 70_000, 1 << 20])
def test_verify_thin_remainders(drawn, V):
    """What is left beside one token that was all but certain: multiples of
    2^-56 up to 2^-46 each, exact in 32 bits, and drawn from."""
    rng = np.random.Generator(np.random.PCG64(V))
    R = 3
    p = np.ldexp(rng.integers(1, 1 << 10, (R, 2, V)).astype(np.float32), -56)
    q = np.ldexp(rng.integers(0, 1 << 8, (R, 2, V)).astype(np.float32), -56)
    sure = rng.integers(0, V, R)
    p[np.arange(R), 0, sure] = np.float32(1 - 2.0 ** -24)
    q[np.arange(R), 0, sure] = 1
    token = np.stack([np.zeros(R), sure], 1).astype(np.int32)
    x = dict(n_nodes=np.full(R, 2), parent=np.tile([-1, 0], (R, 1)).astype(np.int32), token=token, p=torch.tensor(p),
             q=torch.tensor(q) if drawn else None, u_accept=np.ones((R, 2), np.float32), u_sample=rng.random(R, dtype=np.float32))
    check_verify(x)


@pytest.mark.parametrize("dtype,d", KINDS)
def test_a_plan_of_another_rope_theta_is_reported(dtype, d):
    t = Tree(dtype, d=d, lens=(50, 10), T=3, seed=24)
    s = t.session()
    s.desc.rope_theta = 2 * t.theta
    t.check(rows=[], s=s)
    assert s.device_flags() == 32
    s.commit(t.k, t.v, torch.zeros(1, 3, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda"))
    assert s.device_flags() == 32
    s.desc.rope_theta = t.theta
    t.check(s=s)


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_refused_rows_do_not_take_others_along(dtype, d):
    base = dict(dtype=dtype, d=d, lens=(100, 20, 30, 40), T=4, seed=25)
    for what, change, bit in (
            ("nodes beyond the table", dict(n_nodes=[4, 1000, 4]), 64), ("the most nodes", dict(n_nodes=[4, 2 ** 31 - 1, 4]), 64),
            ("a bad parent, on another's tokens", dict(parent=[[-1, 0, 1, 2], [-1, 2, 0, 1], [-1, 0, 0, 0]]), 64),
            ("no block, on another's tokens", dict(tree_block=[1, -1, 3]), 1)):
        t = Tree(**base)
        ts = t.tree_start.copy()
        if "another" in what:
            ts[1] = ts[2] + 1
        s, f = flags_of(t, tree_start=ts, **change)
        assert f == bit, what
        t.tree_block = np.asarray([1, 2, 3], np.int32)
        t.n_nodes = np.clip(t.n_nodes, 0, 4)
        t.parent[1] = [-1, 0, 0, 0]
        t.check(rows=[0, 2], s=s, what=what)
    # trees behind their blocks: the first one at token 0, another row without a block
    t = Tree(in_place=True, **base)
    t.block_len[1] = 0
    t.block_start = np.asarray([200, 0, 20, 60], np.int32)
    t.cap = max(t.cap, 320)
    g = torch.Generator(device="cuda").manual_seed(1)
    t.k, t.v = [torch.randn(t.hkv, t.cap, d, generator=g, device="cuda").to(t.k.dtype) for _ in range(2)]
    t.tree_start = t.block_start[1:] + t.block_len[1:]
    s, f = flags_of(t, tree_block=[1, -1, 3])
    assert f == 1
    t.tree_block = np.asarray([1, 2, 3], np.int32)
    t.check(rows=[0, 2], s=s)


def test_commit_of_one_block_by_the_row_that_may():
    """Two rows of one block: a row whose path is refused has no destination."""
    for bad, n_bad in (([0, 0, -1, -1], 2), ([1, 4, -1, -1], 2), ([0, 1, 2, 3], 5), ([0, 1, 2, 3], -1), ([-1, -1, -1, -1], 1)):
        t = Tree("f32", hq=4, hkv=2, lens=(50, 7, 30), T=4, tree_block=[1, 1], seed=32)
        s = t.session()
        k, v = t.k.clone(), t.v.clone()
        s.commit(k, v, ref.dev([[0, 2, 3, -1], bad]), ref.dev([3, n_bad]))
        assert s.device_flags() == 64, bad
        end, at = int(t.block_start[1] + t.block_len[1]), int(t.tree_start[0])
        for got, x in ((k, t.k), (v, t.v)):
            want = x.clone()
            want[:, end:end + 3] = want[:, [at, at + 2, at + 3]]
            assert torch.equal(bits(got), bits(want)), bad
    # two paths that may both move meet
    t = Tree("f32", hq=4, hkv=2, lens=(50, 7, 30), T=4, tree_block=[1, 1], seed=32)
    s = t.session()
    k = t.k.clone()
    s.commit(k, t.v.clone(), ref.dev([[0, 2, 3, -1], [0, 1, -1, -1]]), ref.dev([3, 2]))
    assert s.device_flags() == 2 and torch.equal(bits(k), bits(t.k))


# ------------------------------------------------- calls with a stream of their own

def busy(stream=None, ms=60):
    """Work that keeps a stream busy for about so long."""
    with torch.cuda.stream(stream or torch.cuda.current_stream()):
        torch.cuda._sleep(int(ms * 1.5e6))


@pytest.mark.parametrize("handle", [False, True])
def test_a_plan_converts_on_its_own_stream(handle):
    """The current stream is busy while a plan on another one converts its
    arrays; the plans before it are still to come when their arrays go."""
    st = torch.cuda.Stream()
    stream = st.cuda_stream if handle else st
    good = [Tree("bf16", lens=(300, 40, 129), T=6, in_place=True, seed=90 + i) for i in range(3)]
    want = []
    for t in good:
        o, l = t.run(t.session())
        want.append(o.clone())
    s = good[0].session()
    arrays = [[ref.dev(x, torch.int64) for x in (t.tree_block, t.n_nodes, t.parent)] for t in good]
    outs = [torch.empty_like(t.q) for t in good]
    torch.cuda.synchronize()
    busy()        # the current stream: what is made there comes late
    busy(st, 30)  # the plans' stream: the host is ahead by all three
    for i, (t, o) in enumerate(zip(good, outs)):
        s.plan(*arrays[i], stream=stream)
        s.decode(t.q, t.k_new, t.v_new, t.k, t.v, out=o, want_lse=False, stream=stream)
        junk = [torch.full((n,), 2 ** 30, dtype=torch.int32, device="cuda") for n in (2, 2, 12, 2) for _ in range(8)]
        del junk
    torch.cuda.synchronize()
    assert s.device_flags() == 0
    for o, w in zip(outs, want):
        assert torch.equal(bits(o), bits(w))


@pytest.mark.parametrize("handle", [False, True])
def test_outputs_do_not_take_memory_that_is_still_in_use(handle):
    """Memory that a caller has given back may still be written by its stream."""
    st = torch.cuda.Stream()
    stream = st.cuda_stream if handle else st
    t = Tree("bf16", lens=(300, 40, 129), T=6, seed=93)
    s = t.session()
    o, l = t.run(s)
    rng = np.random.Generator(np.random.PCG64(93))
    x = draw_verify(rng, 4, 5, 100, "f32", True)
    args = [ref.dev(x["n_nodes"]), ref.dev(x["parent"]), ref.dev(x["token"]), x["p"].cuda(), x["q"].cuda(),
            ref.dev(x["u_accept"], torch.float32), ref.dev(x["u_sample"], torch.float32)]
    verified = [g.clone() for g in engine.tree_verify(*args)]
    torch.cuda.synchronize()
    old = [torch.empty_like(y) for y in (o, l, *verified)]
    busy()
    for y in old:
        y.fill_(7)
    del old, y
    o2, l2 = s.decode(t.q, t.k_new, t.v_new, t.k, t.v, stream=stream)
    got = engine.tree_verify(*args, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(bits(o2), bits(o)) and torch.equal(l2, l)
    for a, b in zip(got, verified):
        assert torch.equal(a, b)


def test_a_session_captured_with_its_plan():
    """plan() and decode() of the session itself in a graph, on arrays of the
    caller's; the session and other sessions go on beside it."""
    t, t2 = (Tree("bf16", lens=(300, 40, 129), T=6, in_place=True, seed=94 + i) for i in range(2))
    want = [x.run(x.session())[0].clone() for x in (t, t2)]
    s = t.session()
    arrays = [ref.dev(x) for x in (t.tree_block, t.n_nodes, t.parent)]
    g, out = torch.cuda.CUDAGraph(), torch.empty_like(t.q)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        s.plan(*arrays)
        s.decode(t.q, t.k_new, t.v_new, t.k, t.v, out=out, want_lse=False)
    mine = (t.q, t.k_new, t.v_new, t.k, t.v, arrays[2])
    first, second = [y.clone() for y in mine], (t2.q, t2.k_new, t2.v_new, t2.k, t2.v, ref.dev(t2.parent))
    for values, w in ((first, want[0]), (second, want[1]), (first, want[0])):
        for a, b in zip(mine, values):
            a.copy_(b)
        out.fill_(1)
        g.replay()
        assert torch.equal(bits(out), bits(w))
    assert s.device_flags() == 0
    del g
    s.plan(*arrays)
    assert torch.equal(bits(s.decode(t.q, t.k_new, t.v_new, t.k, t.v)[0]), bits(want[0]))


# ----------------------------------------------------------- what scores keep

@pytest.mark.parametrize("spread", [1.0, 6.0])
@pytest.mark.parametrize("T,n", [(4, 600), (40, 3000)])
def test_bf16_scores_keep_two_parts_of_a_query(spread, T, n):
    """A turned query is held as two bf16 parts, as the decode holds it: half a
    step twice, 2^-16 of it, and as much again for sums in fp32.  So lse is that
    near, and a weight is off by its own rounding and twice that (a quotient)."""
    t = Tree("bf16", hq=10, hkv=2, lens=(n, 40, 300), T=T, seed=100 + T, scale=spread * 128 ** -0.5)
    t.q_pos = t.q_pos + 100_000
    s = t.session()
    out, lse = t.run(s)
    o, l, absv, reach = ref.attend(
        q=ref.to_np(t.q), k=np.nan_to_num(t.stored(t.k, None)), v=np.nan_to_num(t.stored(t.v, None)), block_start=t.block_start,
        block_len=t.block_len, views=t.view_block, offsets=t.view_offset, q_pos=t.q_pos, tree_block=t.tree_block,
        tree_start=t.tree_start, n_nodes=t.n_nodes, parent=t.parent, heads=t.heads, scale=t.scale, theta=t.theta)
    score = 2.0 ** -15 * reach
    worst = (np.abs(ref.to_np(lse) - l) / (score + 1e-5)).max()
    assert worst <= 1
    step = STEP["bf16"]
    most = step * np.abs(o) + 1.05 * (step + 2 * score[..., None]) * absv + 1e-6
    worst = (np.abs(ref.to_np(out) - o) / most).max()
    assert worst <= 1
