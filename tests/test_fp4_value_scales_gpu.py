"""Decode over 4-bit caches whose value scales span all that the format has (2^-100 to 2^97), zeros
among them: a token's share of the sum does not hang on its values, whatever the others' are.

Scores are known in 64 bits (one element, queries not turned).  Tolerance as in
test_fp4_weights_gpu: 2^-8 of a weight for its parts and its score, 2^-9 for the output's bf16,
and N roundings of 2^-18 of the largest w |v| (a value of zeros takes the place of one of
2^-101).  lse: scores to 2^-12, and 2^-17 for log2 of a scale that is added and taken off again."""
import math

import pytest
import torch

from tests.test_fp4_weights_gpu import TIGHT, decode, exact

pytestmark = pytest.mark.gpu


def tokens(lg, vs):
    """One block: scores lg [n] in units of log2, value scales vs [n], values drawn."""
    n = len(lg)
    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.zeros(1, n, 64, dtype=torch.uint8, device="cuda")
    k[..., 0] = 0x02
    v = torch.randint(0, 256, (1, n, 64), generator=g, device="cuda", dtype=torch.uint8) & 0x88 | 0x22
    v[..., :32] = 0x22
    s = torch.stack([torch.as_tensor(lg).double().cuda() / 16, torch.as_tensor(vs).double().cuda()], -1)[None]
    v[s[..., 1] == 0] = 0
    q = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 16 * math.log(2)
    return q, k, v, s.to(torch.bfloat16)


def check(case):
    q, k, v, s = case
    n = k.shape[1]
    out, lse = decode(q, k, v, s)
    floor = s.clone()
    floor[..., 1] = torch.where(s[..., 1] == 0, 2.0 ** -101, s[..., 1])
    want, lse_want, size, _ = exact(q, s, v, n)
    top = exact(q, floor, v, n)[3]
    bound = TIGHT * size + want.abs() * 2.0 ** -9 + 6 * math.sqrt(n) * 2.0 ** -18 * top[:, None]
    err = (out - want).abs()
    assert (err <= bound).all(), f"{(err / bound).max().item():.3g} of the bound"
    assert (want[:, :64].abs() > bound[:, :64]).all() or not want.any()  # (the bound says something)
    most = (s[..., 0].double() * 16).abs().amax().item()
    assert ((lse - lse_want).abs() <= (most + 1) * 2.0 ** -12 + 2.0 ** -17 + 2.0 ** -19 * lse_want.abs()).all()


LENGTHS = [7, 128, 300, 5000, 60000]  # of one tile, of a few, of many CTAs


@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("e", [97, 70, 40, 10, 0, -9, -40, -63, -80, -100])
def test_zeros_beside_any_scale(n, e):
    vs = torch.full((n,), 2.0 ** e, dtype=torch.float64)
    vs[::2] = 0
    check(tokens(torch.zeros(n), vs))
    vs = torch.full((n,), 2.0 ** e, dtype=torch.float64)
    vs[: n // 2] = 0  # tiles, and CTAs, of nothing else
    check(tokens(torch.zeros(n), vs))
    check(tokens(torch.zeros(n), vs.flip(0)))


@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("lo,hi", [(-70, 64), (-100, 97), (-100, -60), (-20, 97), (-7, 97), (60, 97), (-30, 0)])
@pytest.mark.parametrize("more", [0, 20])
def test_scales_far_apart(n, lo, hi, more):
    """Small values whose weights are 2^more times those of large ones: they are the sum."""
    small = torch.zeros(n, dtype=torch.bool)
    for pick in (slice(0, None, 2), slice(0, n // 2), slice(n // 2, None), slice(n - 1, None)):
        small[:] = False
        small[pick] = True
        lg = torch.where(small, float(more), 0.0)
        vs = torch.where(small, torch.tensor(2.0 ** lo, dtype=torch.float64), torch.tensor(2.0 ** hi, dtype=torch.float64))
        check(tokens(lg, vs))


def test_every_scale_at_once():
    n = 198 * 40
    e = torch.arange(n) % 198 - 100
    g = torch.Generator().manual_seed(1)
    lg = 4 * torch.randn(n, generator=g)
    for order in (torch.arange(n), e.argsort(), e.argsort(descending=True)):
        check(tokens(lg[order], torch.ldexp(torch.ones(n, dtype=torch.float64), e[order])))


def test_lse_does_not_hang_on_values():
    """The same scores over values of ordinary size and of any."""
    n = 3000
    g = torch.Generator().manual_seed(2)
    lg = 3 * torch.randn(n, generator=g)
    e = torch.randint(-100, 98, (n,), generator=g)
    a = decode(*tokens(lg, torch.ones(n, dtype=torch.float64)))[1]
    b = decode(*tokens(lg, torch.ldexp(torch.ones(n, dtype=torch.float64), e)))[1]
    c = decode(*tokens(lg, torch.zeros(n, dtype=torch.float64)))[1]
    assert (a - b).abs().item() <= 2.0 ** -17 and (a - c).abs().item() <= 2.0 ** -17
