"""Decode over 4-bit caches (hw_attn_decode_planned_fp4 and its forms with appends and
view limits) against attention over the decoded, scaled cache in 64 bits.

The bound is that of the arithmetic.  A rotated query element is off by 2^-12 of itself (three
E4M3 parts, half a step 2^-4 each) and 2^-19 of the largest one (where E4M3 runs out
of exponents: 2^-10 beside a largest element of 224 and up), and its angle by 2^-20
(the fast sine); so a score by at most
  ds = scale * sum_i |k_i| ((2^-12 + 2^-20) |q_i| + 2^-18 max|q|),
taken over a row's tokens, and a weight by e^ds.  A weight's two parts add
2^-8 of it, what is below E4M3's steps 2^-18 of the largest one (half a step of the
second part, 2^-14, beside weights of 16 and up), the output its half step 2^-8.  lse
sums weights before they are rounded."""
import numpy as np
import pytest
import torch

from concurrent_shared_kv_gb300 import api, engine
from tests import fp4_ref as F

pytestmark = pytest.mark.gpu


class Case:
    """Blocks laid one behind the other with gaps, views over them, codes drawn."""

    def __init__(self, lens, views, hq, hkv, *, theta=1e6, seed=0, gap=3, limits=None, scale=128 ** -0.5, q_size=1.0,
                 fill=0xff, q_to_kv=None, offsets=None, q_pos=None):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.views, self.hq, self.hkv, self.theta, self.scale = list(lens), views, hq, hkv, theta, scale
        self.limits, self.q_to_kv = limits, q_to_kv
        self.starts, at = [], gap
        for n in self.lens:
            self.starts.append(at)
            at += n + gap
        self.cap, self.R, self.V = at, len(views), max(len(v) for v in views)
        self.views = [list(v) + [-1] * (self.V - len(v)) for v in views]
        self.k = torch.full((hkv, at, 64), fill, dtype=torch.uint8, device="cuda")
        self.v = self.k.clone()
        self.s = torch.full((hkv, at, 2), float("nan"), dtype=torch.bfloat16, device="cuda")  # outside blocks: never used
        for s, n in zip(self.starts, self.lens):
            for pool, i in ((self.k, 0), (self.v, 1)):
                pool[:, s:s + n], self.s[:, s:s + n, i] = F.draw(g, hkv, n, 128)
        self.q = (q_size * torch.randn(self.R, hq, 128, generator=g, device="cuda")).to(torch.bfloat16)
        if offsets is None:
            offsets, ends = [], []
            for view in self.views:
                o, at = [], 0
                for b in view:
                    o.append(at)
                    at += self.lens[b] if b >= 0 else 0
                offsets.append(o)
                ends.append(at)
            q_pos = ends if q_pos is None else q_pos
        self.offsets, self.q_pos = offsets, q_pos

    def session(self):
        t = engine.DecodeSession(n_rows=self.R, n_q_heads=self.hq, n_kv_heads=self.hkv, head_dim=128,
                                 n_blocks=len(self.lens), max_view_blocks=self.V, capacity=self.cap, dtype=torch.bfloat16,
                                 rope_theta=self.theta, scale=self.scale, kv_fp4=True,
                                 view_limits=self.limits is not None)
        t.set_metadata(self.starts, self.lens, self.views, self.offsets, self.q_pos, self.q_to_kv)
        return t

    def run(self, **kw):
        t = self.session()
        if self.limits is None:
            t.plan()
        else:
            t.plan_limited(self.limits)
        out, lse = t.decode_planned_fp4(self.q, self.k, self.v, self.s, **kw)
        assert t.device_flags() == 0
        return out, lse

    def values(self):
        lut = torch.tensor(np.concatenate([F.LEVELS, -F.LEVELS]), device="cuda")

        def of(p, s):
            return torch.stack([lut[(p & 15).long()], lut[(p >> 4).long()]], -1).flatten(-2) * s.double()[..., None]
        return of(self.k, self.s[..., 0]), of(self.v, self.s[..., 1])

    def exact(self, r, k, v):
        """Row r in 64 bits: out [Hq, 128], lse [Hq], the bounds of their errors."""
        freq = torch.tensor([self.theta ** (-i / 64) for i in range(64)], dtype=torch.float64, device="cuda")
        q = self.q[r].double()
        parts, values, sums, sizes = [], [], [], []
        kv = [h // (self.hq // self.hkv) for h in range(self.hq)] if self.q_to_kv is None else list(self.q_to_kv)
        for i, (b, off) in enumerate(zip(self.views[r], self.offsets[r])):
            if b < 0 or self.lens[b] == 0:
                continue
            n = self.lens[b]
            if self.limits is not None and self.limits[r][i] >= 0:
                n = min(n, self.limits[r][i])
            a = (self.q_pos[r] - off) * freq
            x0, x1 = q[:, :64], q[:, 64:]
            t = torch.cat([x0 * a.cos() - x1 * a.sin(), x1 * a.cos() + x0 * a.sin()], -1)
            kb = k[kv, self.starts[b]:self.starts[b] + n]  # [Hq, n, 128]
            reach = torch.cat([(x0 ** 2 + x1 ** 2).sqrt()] * 2, -1)
            parts.append(torch.einsum("hd,hnd->hn", t, kb))
            sums.append(torch.einsum("hd,hnd->hn", t.abs() * 2.0 ** -12 + reach * 2.0 ** -20, kb.abs()))
            sizes.append(kb.abs().sum(-1))
            # (a NaN scale of either kind makes out and lse NaN)
            parts[-1] = parts[-1] + 0 * v[kv, self.starts[b]:self.starts[b] + n].sum(-1)
            values.append(v[kv, self.starts[b]:self.starts[b] + n])
        if not parts or sum(p.shape[1] for p in parts) == 0:
            z = torch.zeros(self.hq, 128, dtype=torch.float64, device="cuda")
            return z, torch.full((self.hq,), -np.inf, dtype=torch.float64, device="cuda"), z, z[:, 0]
        score, vals = torch.cat(parts, -1) * self.scale, torch.cat(values, 1)
        # (a segment's parts share one scale: the largest element of all rows and heads)
        ds = ((torch.cat(sums, -1) + torch.cat(sizes, -1) * self.q[torch.isfinite(self.q)].abs().max().item() * 2.0 ** -18)
              * abs(self.scale)).amax(-1) + 1e-5
        w = torch.softmax(score, -1)
        out = torch.einsum("hn,hnd->hd", w, vals)
        size = torch.einsum("hn,hnd->hd", w, vals.abs())
        # weights small beside the largest w |v| of the row: what their parts leave
        left = (w * vals.abs().amax(-1)).amax(-1, keepdim=True) * 2.0 ** -18 * score.shape[1]
        bound = out.abs() * 2.0 ** -8 + size * (2.0 ** -8 + 2 * torch.expm1(ds)[:, None]) + left + 1e-7
        return out, torch.logsumexp(score, -1), bound, ds + 2.0 ** -19 * (1 + torch.logsumexp(score, -1).abs())

    def check(self, out, lse, rows=None, whole=0.005):
        k, v = self.values()
        for r in range(self.R) if rows is None else rows:
            want, lse_want, bound, lse_bound = self.exact(r, k, v)
            nan = torch.isnan(want)
            assert torch.equal(nan, torch.isnan(out[r])), f"row {r}"
            want, bound = want[~nan], bound[~nan]
            err = (out[r][~nan].double() - want).abs()
            assert (err <= bound).all(), f"row {r}: {(err / bound).max().item():.3g} of the bound"
            # and far inside of it as a whole: the rounding errors are independent
            assert whole is None or err.norm() <= whole * want.norm() + 1e-6, f"row {r}: {(err.norm() / want.norm()).item():.3g}"
            if lse is not None:
                fin = torch.isfinite(lse_want)
                assert torch.equal(fin, torch.isfinite(lse[r]))
                assert torch.equal(lse_want == -np.inf, lse[r] == -np.inf)
                assert ((lse[r].double() - lse_want).abs()[fin] <= lse_bound[fin]).all()


def combined(problems, workers, lens):
    views = []
    for p in range(problems):
        base = p * (workers + 1)
        for w in range(workers):
            views.append([base] + [base + 1 + o for o in range(workers) if o != w] + [base + 1 + w])
    return views


SHAPES = {  # lens, views, hq, hkv
    "one token": ([1], [[0]], 1, 1),
    "one head": ([300], [[0]], 1, 1),
    "two workers": ([256, 32, 40], combined(1, 2, None), 4, 2),
    "ragged tiles": ([129, 127, 1], combined(1, 2, None), 40, 8),
    "four workers": ([2000, 300, 200, 130, 64], combined(1, 4, None), 40, 8),
    "one kv head": ([1000, 50, 60], combined(1, 2, None), 16, 1),
    "no groups": ([700, 90, 33], combined(1, 2, None), 8, 8),
    "32 columns": ([515, 65], [[0, 1]] * 1, 32, 1),
    "column groups": ([700, 100], [[0, 1]] * 9, 40, 8),
    "empty blocks": ([400, 0, 17, 0], combined(1, 3, None), 16, 4),
    "an empty view": ([40, 30], [[0, 1], [-1, -1], [1]], 8, 2),
    "three problems": ([900, 10, 20, 3000, 70, 1, 128, 128, 128], combined(3, 2, None), 32, 8),
}


@pytest.mark.parametrize("what", SHAPES)
def test_decode(what):
    lens, views, hq, hkv = SHAPES[what]
    c = Case(lens, views, hq, hkv, seed=len(what))
    c.check(*c.run())


# ------------------------------------------------------------------- masks

def test_limits():
    """Limits anywhere in the blocks, at tile edges, 0, past the end, of none; rows that
    attend to nothing; and codes and scales of tokens that all limits mask."""
    lens = [700, 129, 64, 3]
    views = [[0, 1], [0, 2], [0, 3], [1, 2], [0, 1, 2, 3], [2, 3], [0]]
    limits = [[128, 1], [129, -1], [127, 2], [0, 0], [500, 500, 0, 1], [0, 64], [-1]]
    limits = [x + [-1] * (4 - len(x)) for x in limits]
    c = Case(lens, views, 16, 4, seed=21, limits=limits)
    out, lse = c.run()
    c.check(out, lse)
    assert (out[3] == 0).all() and (lse[3] == -np.inf).all()


def test_masked_tokens_count_for_nothing():
    """A token with NaN scales: the rows whose limits leave it out are as they were,
    the others NaN, in the heads that share its kv head."""
    lens = [300, 200]
    views, limits = [[0, 1]] * 3, [[299, 150], [299, -1], [-1, 10]]
    c = Case(lens, views, 8, 2, seed=22, limits=limits)
    at = c.starts[0] + 299
    c.s[1, at] = float("nan")
    for h, t in ((0, 150), (0, 199)):
        c.s[h, c.starts[1] + t, t & 1] = float("nan")
    out, lse = c.run()
    c.check(out, lse)
    nan = torch.isnan(out).all(-1)
    assert torch.equal(nan.cpu(), torch.tensor([[False] * 8, [True] * 4 + [False] * 4, [False] * 4 + [True] * 4]))
    assert torch.equal(torch.isnan(lse), nan)


@pytest.mark.parametrize("which", [0, 1])
def test_a_nan_scale_reaches_who_attends(which):
    c = Case([600, 50, 40], combined(1, 2, None) + [[1]], 16, 2, seed=23)
    c.s[1, c.starts[2] + 7, which] = float("nan")
    out, lse = c.run()
    c.check(out, lse)
    assert torch.isnan(out[:2, 8:]).all() and torch.isnan(lse[:2, 8:]).all()
    assert torch.isfinite(out[2]).all() and torch.isfinite(out[:, :8]).all()


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 3e38])
def test_a_bad_query_is_its_own(bad):
    """A query that is not finite (or whose squares are not) is NaN in its row and head
    alone; in segments behind a CTA's first one, too."""
    lens = [2000] + [9] * 60
    views = [[0, 1 + i] for i in range(60)]
    c = Case(lens, views, 8, 4, seed=24)
    bad_rows = [0, 17, 59]
    for r in bad_rows:
        c.q[r, r % 8, 5] = bad
    out, lse = c.run()
    want = torch.zeros(60, 8, dtype=torch.bool)
    for r in bad_rows:
        want[r, r % 8] = True
    assert torch.equal(torch.isnan(out).all(-1).cpu(), want) and torch.equal(torch.isnan(lse).cpu(), want)
    if bad < 1e38:
        return
    c.q = torch.where(c.q.abs() < 1e3, c.q, torch.full_like(c.q, float("nan")))
    c.check(out, None)


# ------------------------------------------------------------------ numbers

def test_zero_values_beside_small_ones():
    """Tokens whose values are all zero weigh in the sum and take no precision from the
    others, however small those are."""
    for small in (1.0, 2.0 ** -12, 2.0 ** -40):
        c = Case([500, 40], [[0, 1], [0]], 8, 2, seed=25)
        c.s[..., 1] *= small
        zero = torch.zeros(c.cap, dtype=torch.bool, device="cuda")
        zero[c.starts[0]:c.starts[0] + 500:3] = True
        zero[c.starts[0]:c.starts[0] + 130] = True  # a whole tile of them
        c.s[:, zero, 1] = 0
        c.v[:, zero] = 0
        out, lse = c.run()
        k, v = c.values()
        for r in range(2):
            want, lse_want, bound, lse_bound = c.exact(r, k, v)
            err = (out[r].double() - want).abs()
            assert (err <= bound).all() and err.norm() <= 0.005 * want.norm()
            assert ((lse[r].double() - lse_want).abs() <= lse_bound).all()


def test_nothing_but_zeros():
    c = Case([300], [[0]], 4, 1, seed=26)
    c.k.zero_(), c.v.zero_(), c.s.zero_()
    out, lse = c.run()
    assert (out == 0).all()
    assert ((lse - np.log(300)).abs() <= 2.0 ** -20 * 6).all()


@pytest.mark.parametrize("spread", [1.0, 2.5])
def test_scales_of_unlike_size(spread):
    c = Case([900, 70, 30], combined(1, 2, None), 40, 8, seed=27)
    c.s[..., 1] *= torch.exp(spread * torch.randn(c.s[..., 1].shape, generator=c.g, device="cuda")).to(torch.bfloat16)
    c.check(*c.run())


@pytest.mark.parametrize("size", [1e-30, 1e-3, 1.0, 30.0])
def test_query_sizes(size):
    c = Case([900, 70, 30], combined(1, 2, None), 16, 8, seed=28, q_size=size)
    c.check(*c.run(), whole=0.005 if size <= 1 else None)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_score_scales(scale):
    c = Case([300, 70], [[0, 1], [1]], 8, 2, seed=29, scale=scale)
    c.check(*c.run(), whole=0.005 if abs(scale) < 0.1 else None)


def test_scores_that_grow():
    """Keys that grow along a long block: the references move again and again."""
    c = Case([60000, 100], [[0, 1], [0]], 16, 4, seed=30)
    c.s[..., 0] *= torch.linspace(0.01, 3, c.cap, device="cuda").to(torch.bfloat16)[None]
    c.check(*c.run(), whole=0.01)


def test_head_maps():
    c = Case([515, 65], [[0, 1], [1], [0]], 8, 2, seed=31, q_to_kv=[1, 0, 0, 1, 1, 0, 1, 0])
    c.check(*c.run())


def test_offsets_past_32_bits():
    """Codes past 2^32 bytes from their pool's start, scales past 2^28."""
    c = Case([1000], [[0]], 8, 8, seed=32, gap=9_000_000)
    out, lse = c.run()
    n = slice(c.starts[0], c.starts[0] + 1000)
    small = Case([1000], [[0]], 8, 8, seed=32, gap=0)
    small.k, small.v, small.s = (x[:, n].contiguous() for x in (c.k, c.v, c.s))
    del c
    small.check(out, lse)


# ------------------------------------------------------------------ appends

APPENDS = {  # lens, views, hq, hkv, (block, position) of each row's token
    "tile edges": ([300, 129, 128, 1, 33], combined(1, 4, None), 8, 2, [(1, 128), (2, 127), (3, 0), (4, 32)]),
    "some rows": ([300, 40, 50], combined(1, 2, None) + [[0]], 16, 4, [(1, 39), (-1, 0), (-1, 5)]),
    "inside a block": ([300, 40], [[0, 1], [1]], 8, 8, [(0, 130), (1, 3)]),
    "into a shared block": ([260] + [20] * 40, [[0, 1 + i] for i in range(40)], 40, 8,
                            [(1 + i, 19) if i else (0, 259) for i in range(40)]),
    "many of a CTA": ([30000] + [1 + i % 3 for i in range(30)], combined(1, 30, None), 2, 2,
                      [(1 + i, i % 3) for i in range(30)]),
}


@pytest.mark.parametrize("what", APPENDS)
def test_appends(what):
    """The new tokens' bits are hw_cache_write's, no other byte changes, and the layer
    attends to them."""
    lens, views, hq, hkv, new = APPENDS[what]
    c = Case(lens, views, hq, hkv, seed=40 + len(what))
    kn, vn = (torch.randn(c.R, hkv, 128, generator=c.g, device="cuda").to(torch.bfloat16) for _ in range(2))
    block, pos = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in zip(*new))
    slot = torch.tensor([c.starts[b] + p if b >= 0 else -1 for b, p in new], dtype=torch.int32, device="cuda")
    want = [c.k.clone(), c.v.clone(), c.s.clone()]
    engine.cache_write(kn, vn, slot, pos, *want[:2], rope_theta=c.theta, kv_scale=want[2])
    t = c.session()
    t.plan_append(block, pos)
    out, lse = t.append_decode_planned_fp4(c.q, kn, vn, c.k, c.v, c.s)
    assert t.device_flags() == 0
    for a, b in zip((c.k, c.v, c.s), want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    c.check(out, lse)
    again = t.decode_planned_fp4(c.q, c.k, c.v, c.s)  # the plan holds without the tokens, too
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_a_bad_append_is_left_out():
    c = Case([300, 40, 50], combined(1, 2, None), 8, 2, seed=50)
    kn = torch.ones(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    before = c.k.clone()
    t = c.session()
    t.plan_append([1, 2], [40, 49])  # the first one lies behind its block
    t.append_decode_planned_fp4(c.q, kn, kn, c.k, c.v, c.s)
    assert t.device_flags() & 2  # HW_DEV_BAD_RANGE
    assert torch.equal(c.k[:, c.starts[1] + 40], before[:, c.starts[1] + 40])
    assert not torch.equal(c.k[:, c.starts[2] + 49], before[:, c.starts[2] + 49])


# --------------------------------------------- streams, graphs, bad calls

def test_layers_early_on_a_stream_and_in_a_graph():
    """A step of three layers with a new token each, eager, on another stream, captured and
    replayed, and with early loads: the same bits."""
    def case(i):
        return Case([3000, 200, 150, 140], combined(1, 3, None), 40, 8, seed=60 + i)
    cases = [case(i) for i in range(3)]
    pos = [n - 1 for n in cases[0].lens[1:]]
    new = [[torch.randn(3, 8, 128, generator=c.g, device="cuda").to(torch.bfloat16) for _ in range(2)] for c in cases]
    saved = [[x.clone() for x in (c.k, c.v, c.s)] for c in cases]

    def step(t, outs, early, stream=None):
        t.plan_append([1, 2, 3], pos, stream=stream)
        for i, (c, n) in enumerate(zip(cases, new)):
            t.append_decode_planned_fp4(c.q, *n, c.k, c.v, c.s, outs[i][0], outs[i][1], early=early and i > 0, stream=stream)

    def buffers():
        return [(torch.full((3, 40, 128), float("nan"), dtype=torch.bfloat16, device="cuda"),
                 torch.full((3, 40), float("nan"), device="cuda")) for _ in cases]

    def restore():
        for c, old in zip(cases, saved):
            for x, y in zip((c.k, c.v, c.s), old):
                x.copy_(y)
        torch.cuda.synchronize()

    t = cases[0].session()
    want = buffers()
    step(t, want, False)
    assert t.device_flags() == 0
    for c, (o, l) in zip(cases, want):
        c.check(o, l)

    def same(got):
        torch.cuda.synchronize()
        assert t.device_flags() == 0
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])

    restore()
    side = torch.cuda.Stream()
    got = buffers()
    side.wait_stream(torch.cuda.current_stream())
    step(t, got, True, side)
    same(got)
    restore()
    got = buffers()
    graph = torch.cuda.CUDAGraph()
    block = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    pos = torch.tensor(pos, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()

    def captured(stream):
        t.plan_append(block, pos, stream=stream)
        for i, (c, n) in enumerate(zip(cases, new)):
            t.append_decode_planned_fp4(c.q, *n, c.k, c.v, c.s, got[i][0], got[i][1], early=i > 0, stream=stream)
    with torch.cuda.graph(graph, stream=side):
        captured(side)
    for _ in range(2):
        restore()
        for o, l in got:
            o.fill_(float("nan")), l.fill_(float("nan"))
        graph.replay()
        same(got)


def test_two_sessions_at_once():
    """Steps of two sessions (workspaces of their own) side by side on two streams."""
    cs = [Case([5000, 40, 30], combined(1, 2, None), 40, 8, seed=70 + i) for i in range(2)]
    ts, outs = [c.session() for c in cs], [[], []]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for t, s in zip(ts, streams):
        t.plan(stream=s)
    for _ in range(20):
        for c, t, s, o in zip(cs, ts, streams, outs):
            o.append(t.decode_planned_fp4(c.q, c.k, c.v, c.s, stream=s))
    torch.cuda.synchronize()
    for c, t, o in zip(cs, ts, outs):
        assert t.device_flags() == 0
        c.check(*o[0])
        assert all(torch.equal(x[0], o[0][0]) and torch.equal(x[1], o[0][1]) for x in o)


def test_outputs_at_any_place():
    """out may start at any element, lse may be left out."""
    c = Case([300, 40], [[0, 1], [1]], 8, 2, seed=80)
    want, _ = c.run()
    flat = torch.full((2 * 8 * 128 + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = flat[1:1 + 2 * 8 * 128].view(2, 8, 128)
    _, lse = c.run(out=out, want_lse=False)
    assert lse is None and torch.equal(out, want) and (flat[0] == 7).all() and (flat[-7:] == 7).all()


def test_no_plan_no_rows_no_blocks():
    c = Case([300, 40], [[0, 1], [1]], 8, 2, seed=81)
    t = c.session()
    out = torch.full((2, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    t.decode_planned_fp4(c.q, c.k, c.v, c.s, out)
    assert t.device_flags() & 32 and (out == 7).all()  # HW_DEV_BAD_PLAN
    empty = Case([], [[-1], [-1]], 8, 2, seed=82)
    out, lse = empty.run()
    assert (out == 0).all() and (lse == -np.inf).all()


def test_refusals_behind_the_workspace():
    """What is checked after the workspace: the places of pools and queries."""
    c = Case([300, 40], [[0, 1], [1]], 8, 2, seed=83)
    t = c.session()
    t.plan()
    out = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")

    def status(q=c.q.data_ptr(), k=c.k.data_ptr(), v=c.v.data_ptr(), s=c.s.data_ptr()):
        with pytest.raises(api.HwError) as e:
            api.attn_decode_planned_fp4(t.desc, q, k, v, s, out, None, t.workspace, t.ws_bytes)
        return e.value.status
    assert status(k=c.k.data_ptr() + 16) == -1 and status(v=c.v.data_ptr() + 16) == -1
    assert status(q=c.q.data_ptr() + 2) == -1 and status(k=0) == -1 and status(s=0) == -1
    assert status(s=c.s.data_ptr() + 2) == -1
    with pytest.raises(api.HwError):
        api.attn_decode_planned_fp4(t.desc, c.q, c.k, c.v, c.s, out, None, t.workspace, 64)
    for bad in ((c.q.float(), c.k, c.v, c.s), (c.q[:1], c.k, c.v, c.s), (c.q, c.k[:1], c.v, c.s), (c.q, c.k, c.v, c.s.float()),
                (c.q, c.k, c.v[:, :, :32], c.s), (c.q, c.k.cpu(), c.v, c.s)):
        with pytest.raises(ValueError):
            t.decode_planned_fp4(*bad)
    assert t.device_flags() == 0


def test_the_same_call_gives_the_same_bits():
    c = Case([20000, 300, 200, 130, 64], combined(1, 4, None), 40, 8, seed=84)
    t = c.session()
    t.plan()
    first = t.decode_planned_fp4(c.q, c.k, c.v, c.s)
    for _ in range(10):
        o = t.decode_planned_fp4(c.q, c.k, c.v, c.s)
        assert torch.equal(o[0], first[0]) and torch.equal(o[1], first[1])


@pytest.mark.parametrize("n_blocks", [0, 2])
def test_a_cache_of_nothing(n_blocks):
    """No blocks, or empty ones, in pools of no tokens, whose addresses are null."""
    none = torch.zeros(2, 0, 64, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2, 0, 2, dtype=torch.bfloat16, device="cuda")
    assert scales.data_ptr() == 0
    for appends in (False, True):
        t = engine.DecodeSession(n_rows=2, n_q_heads=4, n_kv_heads=2, head_dim=128, n_blocks=n_blocks, max_view_blocks=1,
                                 capacity=0, dtype=torch.bfloat16, rope_theta=1e4, kv_fp4=True)
        view = [[0 if n_blocks else -1]] * 2
        t.set_metadata([0] * n_blocks, [0] * n_blocks, view, [[0]] * 2, [0, 0])
        q = torch.ones(2, 4, 128, dtype=torch.bfloat16, device="cuda")
        if appends:
            t.plan_append([-1, -1], [0, 0])
            new = torch.ones(2, 2, 128, dtype=torch.bfloat16, device="cuda")
            out, lse = t.append_decode_planned_fp4(q, new, new, none, none, scales)
        else:
            t.plan()
            out, lse = t.decode_planned_fp4(q, none, none, scales)
        assert t.device_flags() == 0
        assert (out == 0).all() and (lse == -np.inf).all()


@pytest.mark.parametrize("limits", [None, [[250, 100, -1], [0, 300, 7], [300, 0, 0]]])
def test_a_block_twice_in_a_view(limits):
    """A block may stand in a view more than once, at other offsets and under other limits."""
    c = Case([300, 40], [[0, 0, 1], [1, 0, 0], [0, 1, 1]], 8, 2, seed=90, limits=limits,
             offsets=[[0, 300, 600], [0, 40, 1000], [7, 2000, 2100]], q_pos=[640, 1300, 2140])
    c.check(*c.run())


@pytest.mark.parametrize("hq,hkv,rows", [(256, 8, 3), (256, 256, 2), (64, 64, 5), (6, 3, 70)])
def test_many_heads_and_rows(hq, hkv, rows):
    c = Case([400] + [5 + i % 7 for i in range(rows)], [[0, 1 + i] for i in range(rows)], hq, hkv, seed=91)
    c.check(*c.run(), rows=range(0, rows, max(1, rows // 5)))


def test_far_positions():
    """Queries and offsets at both ends of what 32 bits hold."""
    c = Case([300, 40], [[0, 1], [1, 0], [0]], 8, 2, seed=92, theta=1e4,
             offsets=[[2 ** 31 - 400, -2 ** 31], [-5, 2 ** 31 - 1], [-2 ** 31, 0]], q_pos=[2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1])
    # (this reference's angles have 53 bits of up to 2^32 radians; scores are off by 2^-20 of |q| |k| for that)
    c.check(*c.run())


def test_limited_layers_early_and_in_a_graph():
    """Layers of one limited plan with early loads, on a stream and replayed: the same bits."""
    limits = [[2000, 20], [1500, -1], [0, 3], [-1, 0]]
    cases = [Case([3000, 40], [[0, 1]] * 4, 40, 8, seed=93 + i, limits=limits) for i in range(3)]
    t = cases[0].session()
    t.plan_limited(limits)
    want = [t.decode_planned_fp4(c.q, c.k, c.v, c.s) for c in cases]
    for c, w in zip(cases, want):
        c.check(*w)
    got = [(torch.full_like(o, float("nan")), torch.full_like(l, float("nan"))) for o, l in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for i, (c, (o, l)) in enumerate(zip(cases, got)):
            t.decode_planned_fp4(c.q, c.k, c.v, c.s, o, l, early=i > 0, stream=side)
    for _ in range(3):
        for o, l in got:
            o.fill_(float("nan")), l.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert t.device_flags() == 0
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------ all together

def test_a_serving_loop():
    """Prompts written, steps of two workers decoded token by token, their steps committed to
    the common block, the cache forked for a second problem, compacted, and decoded: the pools
    hold what the definitions say (within half a step of the codes), and each decode is
    attention over what the pools hold."""
    L, hkv, hq, cap, theta = 2, 2, 8, 1000, 1e4
    g = torch.Generator(device="cuda").manual_seed(90)

    def bf(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.full((L, hkv, cap, 64), 0xff, dtype=torch.uint8, device="cuda") for _ in range(2))
    s = torch.full((L, hkv, cap, 2), float("nan"), dtype=torch.bfloat16, device="cuda")
    ideal = np.full((2, L, hkv, cap, 128), np.nan)  # what the tokens would be in 64 bits

    def held(layer, h, lo, n):
        return [F.values(p[layer, h, lo:lo + n], s[layer, h, lo:lo + n, i]) for i, p in enumerate((k, v))]

    def agree(lo, n):
        for i in range(2):
            sc = s[..., lo:lo + n, i].cpu().double().numpy()
            got = F.values((k, v)[i][:, :, lo:lo + n], s[:, :, lo:lo + n, i])
            assert (np.abs(got - ideal[i, :, :, lo:lo + n]) <= 1.03 * sc[..., None]).all()
            ideal[i, :, :, lo:lo + n] = got  # what later calls see

    def write(lo, n):
        kn, vn = bf(L, n, hkv, 128), bf(L, n, hkv, 128)
        at = torch.arange(lo, lo + n, dtype=torch.int32, device="cuda")
        engine.cache_write(kn, vn, at, at - lo, k, v, rope_theta=theta, kv_scale=s)
        ideal[0, :, :, lo:lo + n] = F.rotate(kn.cpu().double().numpy(), np.arange(n)[:, None], theta).swapaxes(1, 2)
        ideal[1, :, :, lo:lo + n] = vn.cpu().double().numpy().swapaxes(1, 2)
        agree(lo, n)

    common, w0, w1 = 10, 500, 600
    lens = [200, 20, 30]
    write(common, 200), write(w0, 20), write(w1, 30)

    def decode(starts, lens, views, append=None):
        c = Case.__new__(Case)
        c.lens, c.starts, c.hq, c.hkv, c.theta, c.scale = lens, starts, hq, hkv, theta, 128 ** -0.5
        c.cap, c.R, c.V, c.limits, c.q_to_kv = cap, len(views), len(views[0]), None, None
        c.views, c.q = views, bf(len(views), hq, 128)
        c.offsets, c.q_pos = [], []
        for view in views:
            ends = np.cumsum([0] + [lens[b] for b in view])
            c.offsets.append(ends[:-1].tolist())
            c.q_pos.append(int(ends[-1]))
        t = c.session()
        new = [bf(c.R, hkv, 128) for _ in range(2 * L)]
        if append is None:
            t.plan()
        else:
            t.plan_append(append, [lens[b] - 1 for b in append])
        for layer in range(L):
            c.k, c.v, c.s = k[layer], v[layer], s[layer]
            if append is None:
                out, lse = t.decode_planned_fp4(c.q, c.k, c.v, c.s, early=layer > 0)
            else:
                kn, vn = new[2 * layer:2 * layer + 2]
                out, lse = t.append_decode_planned_fp4(c.q, kn, vn, c.k, c.v, c.s, early=layer > 0)
                for r, b in enumerate(append):
                    at = starts[b] + lens[b] - 1
                    ideal[0, layer, :, at] = F.rotate(kn[r].cpu().double().numpy(), lens[b] - 1, theta)
                    ideal[1, layer, :, at] = vn[r].cpu().double().numpy()
            assert t.device_flags() == 0
            c.check(out, lse)
        if append is not None:
            for b in append:
                agree(starts[b] + lens[b] - 1, 1)

    for _ in range(3):  # tokens
        lens[1] += 1
        lens[2] += 1
        decode([common, w0, w1], lens, [[0, 2, 1], [0, 1, 2]], append=[1, 2])
    # both steps to the end of the common block, one behind the other
    engine.block_commit_fp4(k, v, s, k, v, s, [w0, w1], lens[1:], [common + 200, common + 200 + lens[1]],
                            [200, 200 + lens[1]], rope_theta=theta)
    for lo, n, at in ((w0, lens[1], 200), (w1, lens[2], 200 + lens[1])):
        ideal[0, :, :, common + at:common + at + n] = F.rotate(ideal[0, :, :, lo:lo + n], np.full(n, at), theta)
        ideal[1, :, :, common + at:common + at + n] = ideal[1, :, :, lo:lo + n]
        agree(common + at, n)
    total = 200 + lens[1] + lens[2]
    decode([common], [total], [[0]])
    # a second problem from the same prefix, a token written behind it, the worker blocks dropped
    engine.block_move(k, v, [common], [total], [700], kv_scale=s)
    write(700 + total, 1)  # (at position 0 of a block of its own)
    starts, sizes = [common, 700, 700 + total], [total, total, 1]
    decode(starts, sizes, [[0, 2], [1, 2]])
    before = [[held(layer, h, a, n) for layer in range(L) for h in range(hkv)] for a, n in zip(starts, sizes)]
    now = engine.compact(k, v, starts, sizes, kv_scale=s).tolist()
    assert now == [0, total, 2 * total]
    after = [[held(layer, h, a, n) for layer in range(L) for h in range(hkv)] for a, n in zip(now, sizes)]
    for x, y in zip(before, after):
        for a, b in zip(x, y):
            assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    decode(now, sizes, [[0, 2], [1, 2]])
