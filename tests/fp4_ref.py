"""The 4-bit cache format written out from its definition, in 64 bits, and the
cache calls on host arrays: what the tests compare the library with."""
from __future__ import annotations

import numpy as np
import torch

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16(x):
    """The nearest bf16, as float64 (through fp32, exact for what is used here)."""
    return torch.tensor(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


def scale_of(x):
    """x [..., D] -> scales [...]: bf16(max|x| / 6), 0 below 2^-100, NaN from 2^100 on."""
    with np.errstate(all="ignore"):
        top = np.abs(np.asarray(x, np.float64)).max(-1)
        s = bf16((top.astype(np.float32) / np.float32(6)))
        s = np.where(s < 2.0 ** -100, 0.0, s)
        return np.where(top < 2.0 ** 100, s, np.nan)


def encode(x):
    """x [..., D] (values of fp32) -> (codes [..., D] 0..15, scales [...])."""
    x = np.asarray(x, np.float64)
    s = scale_of(x)
    ok = s > 0
    with np.errstate(all="ignore"):
        r = np.where(ok[..., None], np.abs(x) / np.where(ok, s, 1.0)[..., None], 0.0)
    gap = np.abs(r[..., None] - LEVELS)
    least = gap.min(-1, keepdims=True)
    near = gap == least
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(near.sum(-1) > 1, even.argmax(-1), near.argmax(-1))
    code = code + 8 * np.signbit(x)
    return np.where(ok[..., None], code, 0).astype(np.uint8), s


def decode(codes, s):
    """Codes [..., D] under scales [...] as float64."""
    return np.where(codes >= 8, -1.0, 1.0) * LEVELS[codes & 7] * np.asarray(s, np.float64)[..., None]


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(b):
    return np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], 2 * b.shape[-1])


def rotate(x, pos, theta):
    """x [..., D] float64 rotated at pos (broadcast over the leading dimensions)."""
    half = x.shape[-1] // 2
    freq = np.float64(theta) ** (-np.arange(half) / half)
    a = np.asarray(pos, np.float64)[..., None] * freq
    lo, hi = x[..., :half], x[..., half:]
    return np.concatenate([lo * np.cos(a) - hi * np.sin(a), hi * np.cos(a) + lo * np.sin(a)], -1)


def draw(gen, *shape):
    """Codes of a cache in earnest: tokens of unlike size.  (packed uint8 [..., D/2],
    scales bf16 [...]) as torch tensors on the generator's device."""
    x = torch.randn(shape, generator=gen, device=gen.device)
    x = x * torch.exp(0.4 * torch.randn(shape[:-1], generator=gen, device=gen.device))[..., None]
    s = (x.abs().amax(-1) / 6).to(torch.bfloat16)
    level = torch.tensor(LEVELS, dtype=torch.float32, device=gen.device)
    r = (x.abs() / s.float()[..., None])
    mid = (level[1:] + level[:-1]) / 2
    code = torch.bucketize(r, mid).to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def values(packed, s):
    """float64 numpy values of torch tensors packed [..., D/2], scales [...]."""
    return decode(unpack(packed.cpu().numpy()), s.cpu().double().numpy())
