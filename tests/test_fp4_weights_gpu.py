"""Decode over 4-bit caches: weights far below a row's largest, of which many stand in one
stream of tiles (an attention sink before a long block).

Every head of the case is about a CTA's work, so the sink's reference holds for the whole
block.  Queries and keys have one element, the queries are not turned, so a token's
score is q * level * scale and its weight known in 64 bits.

Tolerance: a weight is held to 2^-8 of itself, the output to 2^-9 (bf16, half a step), and scores to
2^-12 of a score of up to 24 units of log2 (what a query's parts keep): 2^-8 of a weight at most, in all
TIGHT of sum w |v|.  What lies below the second part's steps is rounded up or down, by at most
2^-17 of the largest weight; a sequence that is evenly spread over the token's places decides
which, so N tokens are off by no more than N independent roundings of that size:
6 sqrt(N) 2^-18 of the largest weight, with a standard deviation of half a step."""
import math

import pytest
import torch

from concurrent_shared_kv_gb300 import engine

pytestmark = pytest.mark.gpu
TIGHT = 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -8


def sinks(n, below, spread, where=0, common=1.0):
    """One block of n tokens: the token at `where` has the largest weight and a value of zeros,
    the others are 2^-below of it (log2 with a deviation of `spread`) and have the
    value `common` in the first half of the dimensions, drawn signs in the second."""
    heads = min(torch.cuda.get_device_properties(0).multi_processor_count, 256)
    g = torch.Generator(device="cuda").manual_seed(int(below * 10) + n)
    k = torch.zeros(heads, n, 64, dtype=torch.uint8, device="cuda")
    k[..., 0] = 0x02  # level 1 in element 0
    v = torch.randint(0, 256, (heads, n, 64), generator=g, device="cuda", dtype=torch.uint8) & 0x88 | 0x22
    v[..., :32] = 0x22
    if where is not None:
        v[:, where] = 0
    # scores in units of log2: 24 for the sink, 24 - below - spread * x for the others
    lg = 24.0 - below - spread * torch.randn(heads, n, generator=g, device="cuda").clamp(-4, 4)
    if where is not None:
        lg[:, where] = 24.0
    s = torch.empty(heads, n, 2, device="cuda")
    s[..., 0] = lg / 16
    s[..., 1] = common
    if where is not None:
        s[:, where, 1] = 1.0
    s = s.to(torch.bfloat16)
    q = torch.zeros(1, heads, 128, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 16 * math.log(2)
    return q, k, v, s


def decode(q, k, v, s, limit=None):
    heads, n = k.shape[:2]
    t = engine.DecodeSession(n_rows=1, n_q_heads=heads, n_kv_heads=heads, head_dim=128, n_blocks=1, max_view_blocks=1,
                             capacity=n, dtype=torch.bfloat16, rope_theta=1e4, scale=1.0, kv_fp4=True,
                             view_limits=limit is not None)
    t.set_metadata([0], [n], [[0]], [[0]], [0])
    t.plan() if limit is None else t.plan_limited([[limit]])
    out, lse = t.decode_planned_fp4(q, k, v, s)
    assert t.device_flags() == 0
    return out[0].double(), lse[0].double()


def exact(q, s, v, upto):
    """out, lse, sum w |v|, the largest w |v|'s weight of all (sum of weights 1)."""
    score = q[0, :, :1].double() * s[:, :upto, 0].double()
    w = torch.softmax(score, -1)
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    out, size = [], []
    for h in range(s.shape[0]):
        x = torch.stack([lut[(v[h, :upto] & 15).long()], lut[(v[h, :upto] >> 4).long()]], -1).flatten(-2)
        x = x * s[h, :upto, 1:].double()
        out.append(w[h] @ x)
        size.append(w[h] @ x.abs())
    return torch.stack(out), torch.logsumexp(score, -1), torch.stack(size), (w * s[:, :upto, 1].double()).amax(-1)


def check(case, limit=None):
    q, k, v, s = case
    n = k.shape[1] if limit is None else limit
    out, lse = decode(q, k, v, s, limit)
    want, lse_want, size, top = exact(q, s, v, n)
    err = (out - want).abs()
    bound = TIGHT * size + want.abs() * 2.0 ** -9 + 6 * math.sqrt(n) * 2.0 ** -18 * top[:, None]
    assert (err <= bound).all(), f"{(err / bound).max().item():.3g} of the bound, off by {err.max().item():.3g}"
    # the mass behind the sink, over all heads: unbiased
    mean = ((out - want)[:, :64].mean() / want[:, :64].mean()).abs().item()
    assert mean <= TIGHT + 6 * math.sqrt(n) * 2.0 ** -18 * (top.mean() / want[:, :64].mean()).item()
    assert ((lse - lse_want).abs() <= 24 * 2.0 ** -12 + 2.0 ** -19 * (1 + lse_want.abs())).all()


@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("below", [6, 10, 12.3, 14, 14.6, 15, 16, 17.5])
def test_a_sink_before_many_small_weights(below, spread):
    check(sinks(20000, below, spread))


@pytest.mark.parametrize("n,where", [(300, 0), (129, 128), (4097, 4096), (20000, 9999), (1, None), (257, None)])
def test_sinks_at_other_places(n, where):
    check(sinks(n, 14, 1.0, where))


def test_small_values_beside_one_large():
    """The value's scale is part of the weight: a large value takes the sink's place."""
    q, k, v, s = sinks(20000, 3, 1.0)
    v[:, 0] = 0x22
    s[:, 0, 1] = 2048.0
    check((q, k, v, s))


def test_masked_tokens_stay_out():
    """Tokens behind a limit have weights of exactly zero, whatever the rounding adds to small ones."""
    q, k, v, s = sinks(5000, 14, 1.0)
    v[:, 3000:] = 0x77
    s[:, 3000:, 1] = 2.0 ** 60
    check((q, k, v, s), limit=3000)
