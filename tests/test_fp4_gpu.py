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
            values.append(v[kv, self.starts[b]:self.starts[b] + n])
        if not parts or sum(p.shape[1] for p in parts) == 0:
            z = torch.zeros(self.hq, 128, dtype=torch.float64, device="cuda")
            return z, torch.full((self.hq,), -np.inf, dtype=torch.float64, device="cuda"), z, z[:, 0]
        score, vals = torch.cat(parts, -1) * self.scale, torch.cat(values, 1)
        # (a segment's parts share one scale: the largest element of all rows and heads)
        ds = ((torch.cat(sums, -1) + torch.cat(sizes, -1) * self.q.abs().max().item() * 2.0 ** -18)
              * abs(self.scale)).amax(-1) + 1e-5
        w = torch.softmax(score, -1)
        out = torch.einsum("hn,hnd->hd", w, vals)
        size = torch.einsum("hn,hnd->hd", w, vals.abs())
        # weights small beside the largest w |v| of the row: what their parts leave
        left = (w * vals.abs().amax(-1)).amax(-1, keepdim=True) * 2.0 ** -18 * score.shape[1]
        bound = out.abs() * 2.0 ** -8 + size * (2.0 ** -8 + 2 * torch.expm1(ds)[:, None]) + left + 1e-7
        return out, torch.logsumexp(score, -1), bound, ds + 2.0 ** -19 * (1 + torch.logsumexp(score, -1).abs())

    def check(self, out, lse, rows=None):
        k, v = self.values()
        for r in range(self.R) if rows is None else rows:
            want, lse_want, bound, lse_bound = self.exact(r, k, v)
            err = (out[r].double() - want).abs()
            assert (err <= bound).all(), f"row {r}: {(err / bound).max().item():.3g} of the bound"
            # and far inside of it as a whole: the rounding errors are independent
            assert err.norm() <= 0.005 * want.norm() + 1e-6, f"row {r}: {(err.norm() / want.norm()).item():.3g}"
            if lse is not None:
                fin = torch.isfinite(lse_want)
                assert torch.equal(fin, torch.isfinite(lse[r]))
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
